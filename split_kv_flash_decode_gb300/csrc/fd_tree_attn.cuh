// Attention of drafted tokens over the cache (fd_tree_decode) on the fifth-generation tensor cores.
//
// All query rows of a (sequence, KV head), its drafted tokens times the heads of its group, meet every K and V
// row, so the work is two matrix products per tile of 128 tokens: S = Q K^T (rows on M, tokens on N) and
// O += P V, with the online softmax between them.  A row is a lane of tensor memory and belongs to one
// thread: no shuffle is needed for its maximum or its sum.  Rows are padded to 128, which costs nothing
// while HBM is the bound (the two products of a tile take a third of the time that its bytes take).
//
// One CTA per SM runs through an equal share of the tiles of all items (an item: a KV head of a sequence and up
// to 256 of its query rows).  Two groups of four softmax warps work in turn, so that the tensor cores have one
// group's products while the other computes its weights: they take the two row tiles of an item, or, of an
// item with one row tile, alternate tiles of tokens, whose two results they merge at its end.  An item that
// several CTAs share leaves fp32 records (m, l, O), which a second launch combines: no CTA waits for
// another.  (The records of an item that one CTA had alone are never written.)
//
// What bounds it, at 8 KV heads of 128 elements: 16-bit caches and one row tile HBM, most of the time (64 x 8192 tokens, 16
// drafts, groups of 4: 326 to 339 us from box to box, 6.4 to 6.6 TB/s, where a decode reads the same bytes in 303; 32768
// tokens 26.7 us, with the first loads, the records and their combination around 20 us of stream).  Two row tiles: the
// products and the shared memory that feeds them (32768 tokens, 64 drafts, groups of 8: 81 us, 848 TFLOP/s).  8- and 4-bit
// caches: the way of a tile through a converter team, about 1800 clocks from its load's arrival to its operand's (4 bits,
// 131072 tokens, 24 drafts, groups of 8: 131 us, 787 TFLOP/s), and over pages of 16 tokens the issue of the loads, 70 to
// 100 ns a box (E4M3, 64 x 4096 tokens, 5 drafts, groups of 4: 175 us; 127 without pages).  Tiles whose tokens the two
// groups split (S twice in tensor memory): equal over 16 bits, 10 to 22 % slower over the others.
//
// Weights are rounded once to 16 bits, over bf16 caches to two parts of 8 bits.  Two parts of fp16 as well (22 bits) would
// take the error of an fp16 output from 2.8e-4 to 2.1e-4 of it, and 189 instead of 176 us of this E4M3 batch, 172 instead of
// 131 of these 4 bits, 1115 instead of 863 of 32 x 32768 tokens with 64 drafts over f16.
//
// Warps: 0-3 and 4-7 softmax, 8 issues the products, 9 the TMA loads, 10 and 11 bring the next item's queries in, and
// over 8- and 4-bit caches 12 on widen the stored rows to fp16 in the layout that the products read.
#pragma once

#include "fd_kernel.cuh"
#include "fd_tree.h"

namespace fd {
namespace tree {

constexpr int kMmaWarp = 8, kLoadWarp = 9, kQueryWarp = 10, kQueryWarps = 2, kConvertWarp = 12;
FD_HD constexpr int convert_warps(int kv) { return kv == kKv16 ? 0 : 4; }
FD_HD constexpr int threads(int kv) { return 32 * (kConvertWarp + convert_warps(kv)); }
// Registers per thread: at launch (what the compiler takes for that many threads), then softmax, warps 8-11, and
// converters.  A softmax thread holds a row's 128 scores.
FD_HD constexpr int launch_regs(int kv) { return kv == kKv16 ? 168 : 128; }
FD_HD constexpr int softmax_regs(int kv) { return kv == kKv16 ? 216 : 192; }
FD_HD constexpr int other_regs(int kv) { return kv == kKv16 ? 72 : 56; }
constexpr int kConvertRegs = 72;
FD_HD constexpr bool regs_fit(int kv) {
  return 256 * softmax_regs(kv) + 128 * other_regs(kv) + 32 * convert_warps(kv) * kConvertRegs <= threads(kv) * launch_regs(kv);
}
static_assert(regs_fit(kKv16) && regs_fit(kKvE4m3) && regs_fit(kKvE2m1), "setmaxnreg would wait forever");
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Tensor memory, all of it (so that its addresses begin at 0): S (and P in its place) of the two groups, then their O.
constexpr uint32_t kTmemAll = 512, kTmemS = 128, kTmemO = 256;
constexpr int kMaxOperandSlots = 4;  // of 8- and 4-bit caches
constexpr int kPrefetch = 4;         // operand tiles that a CTA brings into L2 ahead of its turn
// Weights are held as 2^(their exponent + this).  A weight reaches 2^kRescaleThreshold, so fp16 weights can use 7 powers
// more, up to 2^15: they are then normal numbers (11 bits) down to 2^-21 of the maximum in use, and off by at most 2^-32
// of it below.  (As they are, a weight of 2^-25 was 0 in the product and still counted in the sum: 128K such tokens
// behind one that leads were lost, 0.4 % of the row.)  bf16 has fp32's exponents.
template <typename Op>
FD_HD constexpr float weight_exponent() {
  return std::is_same<Op, __half>::value ? 7.f : 0.f;
}
static_assert(dev::kRescaleThreshold + 7 <= 15, "fp16 weights stay finite");

// ------------------------------------------------------------------ primitives

__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]; A's 16-bit elements lie in pairs, row by row in the lanes.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Two fp32 values in one register pair.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// A place in a ring of slots, and the parity of its barriers' phase.
struct Place {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ void advance(uint32_t by, uint32_t slots) {
    slot += by;
    if (slot >= slots) {
      slot -= slots;
      parity ^= 1;
    }
  }
};
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
  return yes != 0;
}

// ------------------------------------------------------------------ the work of a CTA

// Tiles [tile0, tile0 + nt) of an item.
struct Portion {
  int b, kvh, r0, L, tile0, nt;
  int16_t rows, n, row_tile;  // row_tile: rows of a row tile
  bool two;    // two row tiles; else one, and the groups take alternate tiles of tokens
  bool whole;  // all tiles of the item
  bool slot;   // the CTA's record: 0 of the item it goes on with, 1 of the item it leaves unfinished
  __device__ __forceinline__ int jobs() const { return two ? 2 * nt : nt; }
  __device__ __forceinline__ int tile_of(int job) const { return two ? job >> 1 : job; }
  // Place of a tile's V among the portion's 2 nt loads, which come in the order in which the products want them.
  __device__ __forceinline__ int seq_v(int t) const { return two || t == nt - 1 ? 2 * t + 1 : 2 * t + 2; }
  // The tile and kind of load s.
  __device__ __forceinline__ bool is_v(int s) const { return two || s == 2 * nt - 1 ? s & 1 : s != 0 && !(s & 1); }
  __device__ __forceinline__ int load_tile(int s) const {
    return two || s == 2 * nt - 1 ? s >> 1 : s == 0 ? 0 : s & 1 ? (s + 1) >> 1 : (s >> 1) - 1;
  }
};

// The portions of a run of units, in order; the same in every warp.
struct Cursor {
  int u, u1, b;
  Cursor() = default;
  __device__ __forceinline__ Cursor(const TreeParams& p, int cta) {
    u = tree_run_begin(p, cta);
    u1 = tree_run_begin(p, cta + 1);
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.unit_base[mid] <= u) lo = mid; else hi = mid;
    }
    b = lo;
  }
  __device__ __forceinline__ bool next(const TreeParams& p, Portion& o) {
    while (u < u1) {
      while (p.unit_base[b + 1] <= u) ++b;
      o.b = b;
      o.L = p.len[b];
      o.n = p.cu_q[b + 1] - p.cu_q[b];
      const int tiles = tree_tiles(o.L), per = tree_item_units(p, tiles), rows = o.n * p.G, groups = tree_groups(rows);
      const int at = u - p.unit_base[b], item = at / per, off = at - item * per;
      const int end = min(u1 - u + off, per);
      u += end - off;
      const int lo = p.whole_items ? 0 : max(0, off - p.item_units);
      const int hi = p.whole_items ? tiles : max(0, end - p.item_units);
      if (hi <= lo) continue;
      o.kvh = item / groups;
      o.r0 = (item - o.kvh * groups) * kTreeRows;
      o.rows = min(rows - o.r0, kTreeRows);
      o.two = o.rows > kTreeTile;
      o.row_tile = o.two ? (o.rows / 2 + 31) / 32 * 32 : kTreeTile;
      if (o.two && o.row_tile * 2 < o.rows) o.row_tile += 32;
      o.tile0 = lo;
      o.nt = hi - lo;
      o.whole = lo == 0 && hi == tiles;
      o.slot = lo == 0;
      return true;
    }
    return false;
  }
};

// Nodes of a sequence as bits.
__device__ __forceinline__ uint64_t all_nodes(int n) { return n >= 64 ? ~0ull : (1ull << n) - 1; }
// Of a tile's columns 32 k .. 32 k + 31, those that a token sees: the columns before `off`, where the drafted rows
// begin, and the nodes of its mask behind.
__device__ __forceinline__ uint32_t seen(uint64_t mask, int off, int k) {
  const int lim = off - 32 * k;
  uint32_t v = lim >= 32 ? ~0u : lim > 0 ? (1u << lim) - 1 : 0u;
  if (lim <= 0 && lim > -64) v |= (uint32_t)(mask >> -lim);
  else if (lim > 0 && lim < 32) v |= (uint32_t)(mask << lim);
  return v;
}
// The nodes that any token of the sequence sees: what a lane of a whole warp looks at, and all of them together.
__device__ __forceinline__ uint64_t seen_by_lane(const TreeParams& p, int b, int n) {
  if (p.mask == nullptr) return all_nodes(n);
  const int lane = threadIdx.x & 31;
  uint64_t m = lane < n ? p.mask[p.cu_q[b] + lane] : 0;
  if (lane + 32 < n) m |= p.mask[p.cu_q[b] + lane + 32];
  return m & all_nodes(n);
}
__device__ __forceinline__ uint64_t seen_by_any(uint64_t m) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m |= __shfl_xor_sync(0xffffffffu, m, off);
  return m;
}

// Waits for a barrier's phase.  Where that takes over a second the CTA is given up: the status word and NaN in its rows say
// so, and no later wait of the CTA waits.
struct Waiter {
  volatile int* dead;
  uint32_t* status;
  __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) const {
    if (dev::mbar_try_wait(bar, parity)) return;
    slow(bar, parity);
  }
  __device__ __forceinline__ void slow(uint32_t bar, uint32_t parity) const {
    const uint64_t start = dev::global_timer_ns();
    while (!*dead) {
#pragma unroll 1
      for (int i = 0; i < 64; ++i)
        if (dev::mbar_try_wait(bar, parity)) return;
      if (dev::global_timer_ns() - start > dev::kWaitLimitNs) {
        *dead = 1;
        if (status != nullptr) atomicOr(status, FD_TREE_TIMEOUT);
      }
    }
  }
};

// ------------------------------------------------------------------ softmax

// A row's weights of one tile, 2^(weight_exponent + score - maximum in use), and their sum l; m is a score, without the
// scale.  ts, to: its lane's S (which its weights replace) and O; first: O holds nothing yet.
template <int D, typename Op>
__device__ __forceinline__ void weigh(uint32_t ts, uint32_t to, bool edge, uint64_t mask, int off, float scale, bool mine,
                                      bool first, float& m, float& l) {
  constexpr bool kBf16 = std::is_same<Op, __nv_bfloat16>::value;
  uint32_t x[128];
#pragma unroll
  for (int c = 0; c < 4; ++c) ld32(ts + 32 * c, x + 32 * c);
  tc::wait_ld();
  if (edge) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t v = seen(mask, off, c);
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (!(v >> k & 1)) x[32 * c + k] = 0xff800000u;
    }
  }
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int k = 0; k < 128; k += 8)
#pragma unroll
    for (int c = 0; c < 4; ++c) mx[c] = max3(mx[c], __uint_as_float(x[k + 2 * c]), __uint_as_float(x[k + 2 * c + 1]));
  const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
  // A row's maximum in use moves only when its weight grew by more than 2^8, which is rare.
  const bool grew = mine && (top - m) * scale > dev::kRescaleThreshold;
  if (__any_sync(0xffffffffu, grew)) {
    const float coef = !grew ? 1.f : m == -INFINITY ? 0.f : dev::ex2((m - top) * scale);
    if (grew) m = top;
    l *= coef;
    if (!first) {  // the group's earlier products are done: this tile's scores were committed behind them
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t y[32];
        ld32(to + c, y);
        tc::wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * coef);
        st32(to + c, y);
      }
    }
  }
  const float mm = m == -INFINITY ? 0.f : m;
  constexpr float kUp = weight_exponent<Op>();
  const uint64_t scale2 = pair(scale, scale), minus2 = pair(-mm, -mm), up2 = pair(kUp, kUp);
  uint64_t sum[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t y[32];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      // Difference, then product: the largest score minus the maximum in use is then exact, however large both are.  (A
      // product and a difference behind it become one instruction, rounding modes or not, which rounds m alone.)
      const uint64_t less = add_pair(pair(__uint_as_float(x[32 * c + 2 * k]), __uint_as_float(x[32 * c + 2 * k + 1])), minus2);
      const float2 e = unpair(kUp != 0.f ? fma_pair(less, scale2, up2) : mul_pair(less, scale2));
      const float f = dev::ex2(e.x), g = dev::ex2(e.y);
      const uint64_t fg = pair(f, g);
      sum[k & 1] = add_pair(sum[k & 1], fg);
      y[k] = dev::pack2<Op>(f, g);
      if constexpr (kBf16) {
        const float2 h = dev::Elem<Op>::to_f2(y[k]);
        const float2 rest = unpair(add_pair(fg, pair(-h.x, -h.y)));
        y[16 + k] = dev::pack2<Op>(rest.x, rest.y);
      }
    }
    // The weights lie where their scores lay: the scores are all read.
    if constexpr (kBf16) st32(ts + 32 * c, y);
    else st16(ts + 32 * c, y);
  }
  const float2 s2 = unpair(add_pair(sum[0], sum[1]));
  l += s2.x + s2.y;
}

// A row's O goes on outside of tensor memory: sums = coef x sums + O; or, at the end (`back`), O += coef x sums.  Where coef
// is 0 there are no sums yet, or none that count.  A call, once in 64 tiles: in line it made the loop around it slower (64 x
// 32K tokens of 4 bits: 1278 us; 1220 so, and 1150 without it).
template <int D>
__device__ __noinline__ void move_sums(uint32_t to, float* sums, float coef, bool back) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float4 o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      o[k] = coef != 0.f ? __ldcg(reinterpret_cast<const float4*>(sums + (c + 4 * k) * kTreeTile)) : make_float4(0.f, 0.f, 0.f, 0.f);
    __syncwarp();
    uint32_t y[32];
    ld32(to + c, y);
    tc::wait_ld();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      o[k].x = fmaf(coef, o[k].x, __uint_as_float(y[4 * k]));
      o[k].y = fmaf(coef, o[k].y, __uint_as_float(y[4 * k + 1]));
      o[k].z = fmaf(coef, o[k].z, __uint_as_float(y[4 * k + 2]));
      o[k].w = fmaf(coef, o[k].w, __uint_as_float(y[4 * k + 3]));
    }
    if (back) {
#pragma unroll
      for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(k % 4 == 0 ? o[k / 4].x : k % 4 == 1 ? o[k / 4].y : k % 4 == 2 ? o[k / 4].z : o[k / 4].w);
      st32(to + c, y);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) __stcg(reinterpret_cast<float4*>(sums + (c + 4 * k) * kTreeTile), o[k]);
    }
  }
  tc::wait_st();
}

// ------------------------------------------------------------------ the kernel

// What a CTA that was given up leaves: NaN in all rows of its portions that are its own, NaN records of the others (which
// make their rows NaN).  A thread takes a row of the 256 that an item can have.
template <int D>
__device__ __noinline__ void leave_nan(const TreeParams& p) {
  const float nan = __int_as_float(0x7fffffff);
  const int row = threadIdx.x;
  Cursor cur(p, blockIdx.x);
  Portion o;
  while (cur.next(p, o)) {
    if (row >= o.rows) continue;
    if (!o.whole) {
      __stcg(p.part + (int64_t)(2 * blockIdx.x + o.slot) * tree_record_floats(D, p.rec_rows) + row, nan);
      continue;
    }
    const int R = o.r0 + row, t = R / p.G;
    const int64_t at = (int64_t)(p.cu_q[o.b] + t) * p.Hq + o.kvh * p.G + (R - t * p.G);
    uint4* out = static_cast<uint4*>(p.out) + at * (D / 8);
    for (int c = 0; c < D / 8; ++c) out[c] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);  // fp16's, bf16's
    if (p.lse != nullptr) p.lse[at] = nan;
  }
}

// kLong: some portion is longer than what a group's products may add up to in tensor memory (tree_sum_tiles).
template <typename T, int D, int KV, bool kLong>
__global__ void __launch_bounds__(threads(KV), 1) fd_tree_kernel(const __grid_constant__ TreeParams p) {
  // Operands: bf16 over a bf16 cache, else fp16.
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value && KV == kKv16;
  using Op = typename std::conditional<kBf16, __nv_bfloat16, __half>::type;
  constexpr bool kScaledQ = std::is_same<T, __nv_bfloat16>::value && !kBf16;
  constexpr int kOperand = tree_operand_bytes(D), kRaw = tree_raw_bytes(KV, D), kHalf = kTreeTile * 128;
  constexpr int CPR = D / 8;  // 16-byte chunks of a row
  extern __shared__ __align__(1024) uint8_t smem[];
  const int q_tiles = p.q_tiles, nslot = tree_slots(KV, D, q_tiles), nraw = tree_raw_slots(KV, D, q_tiles);
  uint8_t* slots = smem + q_tiles * kOperand;
  uint8_t* raws = slots + nslot * kOperand;
  uint8_t* meta = smem + kTreeSmemTiles;
  // The loads' ring (16 bits: the operand slots themselves), then the operand slots of other caches.
  const uint32_t full0 = dev::smem_addr(meta), empty0 = full0 + 8 * kTreeMaxSlots;
  const uint32_t wide0 = empty0 + 8 * kTreeMaxSlots;
  const uint32_t op_full0 = KV == kKv16 ? full0 : wide0;
  const uint32_t op_empty0 = KV == kKv16 ? empty0 : wide0 + 8 * kMaxOperandSlots;
  const uint32_t s_full0 = wide0 + 16 * kMaxOperandSlots, p_ready0 = s_full0 + 16, o_full0 = p_ready0 + 16,
                 q_full0 = o_full0 + 16, q_empty = q_full0 + 16;
  constexpr int kBars = 8 * (2 * kTreeMaxSlots + 2 * kMaxOperandSlots + 9);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(meta + kBars);
  int* dead = reinterpret_cast<int*>(meta + kBars + 4);
  Portion* said = reinterpret_cast<Portion*>(meta + kBars + 8);  // [3]: portion k is in place k % 3; nt = 0: the end
  int8_t* q_exp = reinterpret_cast<int8_t*>(said + 3);           // [2][kTreeRows]: the power of two taken out of a query row
  float* ml = reinterpret_cast<float*>(meta + kTreeMetaBytes - 2048);  // [2][128][2]: the groups' m and l at an item's end
  static_assert(kBars + 8 + 3 * sizeof(Portion) + 2 * kTreeRows + 2048 <= kTreeMetaBytes, "meta");
  const int nload = KV == kKv16 ? nslot : nraw;  // slots of the loads' ring
  // O begins anew in tensor memory with a group's i-th tile of a portion where i & kSumMask == 0, but with the last: there
  // it takes back what has gone on outside.
  constexpr int kSumMask = kLong ? tree_sum_tiles(kBf16) - 1 : -1;
  auto begins_anew = [](int job, int jobs) { return kLong ? ((job >> 1) & kSumMask) == 0 && (job < 2 || job + 2 < jobs) : job < 2; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  dev::pdl_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < nload; ++s) {
      dev::mbar_init(full0 + 8 * s, 1);
      dev::mbar_init(empty0 + 8 * s, KV == kKv16 ? 1 : convert_warps(KV) / 2);
    }
    if (KV != kKv16)
      for (int s = 0; s < nslot; ++s) {
        dev::mbar_init(op_full0 + 8 * s, convert_warps(KV) / 2);
        dev::mbar_init(op_empty0 + 8 * s, 1);
      }
    for (int w = 0; w < 2; ++w) {
      dev::mbar_init(s_full0 + 8 * w, 1);
      dev::mbar_init(p_ready0 + 8 * w, 4);
      dev::mbar_init(o_full0 + 8 * w, 1);
    }
    dev::mbar_init(q_full0, kQueryWarps);
    dev::mbar_init(q_full0 + 8, kQueryWarps);
    dev::mbar_init(q_empty, 1);
    dev::fence_mbar_init();
    *dead = 0;
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(dev::smem_addr(tmem_slot), kTmemAll);
    tc::tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    dev::prefetch_tensormap(&p.tm_k);
    dev::prefetch_tensormap(&p.tm_v);
  }
  // What the parameters alone say is worked out ahead of the wait for the kernels before.
  Cursor cur;
  Portion o = {};
  bool more = false;
  if (warp >= kLoadWarp) {
    cur = Cursor(p, blockIdx.x);
    more = cur.next(p, o);
    if (!more) o = Portion{};  // a run may lie within what an item costs beyond its tiles
    if (warp == kQueryWarp && lane == 0) said[0] = o;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const Waiter wait{dead, p.status};

  // Writes query rows of portion q: chunks of 16 bytes, `step` threads, the first of them `from`.
  auto put_queries = [&](const Portion& q, int from, int step, int parity) {
    constexpr int kBatch = KV == kKv16 ? 4 : 2;
    const int total = q.rows * CPR, G = p.G;
    const T* src = reinterpret_cast<const T*>(p.q) + ((int64_t)p.cu_q[q.b] * p.Hq + q.kvh * G) * D;
    for (int c0 = from;; c0 += kBatch * step) {
      uint4 x[kBatch];
      int64_t at[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int c = c0 + k * step, gr = c / CPR, R = q.r0 + gr, t = R / G;
        at[k] = ((int64_t)t * p.Hq + (R - t * G)) * D + (c - gr * CPR) * 8;
      }
      if (c0 == from && parity < 0) dev::pdl_wait();
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (c0 + k * step < total) x[k] = *reinterpret_cast<const uint4*>(src + at[k]);
      // Portions but the first: the last products with Q's old rows are done.  (Threads without a chunk wait too.)
      if (c0 == from && parity >= 0) wait(q_empty, parity & 1);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int c = c0 + k * step;
        if (c < total) {
          const int gr = c / CPR, ch = c - gr * CPR;
          if constexpr (kScaledQ) {
            // bf16 into fp16 by a power of two for each row that brings its largest value below 2^15.
            float f[8];
            dev::unpack8<T>(x[k], f);
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
            const uint32_t lanes_here = ((1u << CPR) - 1) << (lane & ~(CPR - 1));  // a row's: CPR divides every bound
#pragma unroll
            for (int off = 1; off < CPR; off <<= 1) m = fmaxf(m, __shfl_xor_sync(lanes_here, m, off));
            const int e = (int)(__float_as_uint(m) >> 23);    // 2^(e - 127) <= m
            const int up = e == 0 || e == 255 ? 0 : min(141 - e, 100);
            const float s = __int_as_float((127 + up) << 23);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= s;
            x[k] = make_uint4(dev::pack2<__half>(f[0], f[1]), dev::pack2<__half>(f[2], f[3]),
                              dev::pack2<__half>(f[4], f[5]), dev::pack2<__half>(f[6], f[7]));
            if (ch == 0) q_exp[((parity + 1) & 1) * kTreeRows + gr] = (int8_t)-up;
          }
          const int tile = q.two && gr >= q.row_tile ? 1 : 0, r = gr - tile * q.row_tile;
          *reinterpret_cast<uint4*>(smem + tile * kOperand + (ch >> 3) * kHalf + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = x[k];
        }
      }
      if (c0 + kBatch * step >= total) break;
    }
    tc::fence_proxy_async_smem();
  };

  if (warp < kMmaWarp) {
    regs_inc<softmax_regs(KV)>();
    // ---------------- softmax
    const int w = warp >> 2, wl = tid & 127;             // group, and thread in it: the row in its tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = lanes + w * kTmemS, to = lanes + kTmemO + w * kTmemS;
    uint32_t base = 0, s_phase = 0, o_phase[2] = {0, 0};
    // The m and l of sums outside of tensor memory lie where the item's end leaves its own.
    float2* const own_ml = reinterpret_cast<float2*>(ml + 256 * w + 2 * wl);
    // The first item's queries, for which everybody waits, are brought in by all.
    put_queries(said[0], tid, 256 + 32 * kQueryWarps, -1);
    tc::named_sync(2, 256 + 32 * kQueryWarps);
    for (uint32_t nth = 0;; ++nth) {
      const Portion o = said[nth % 3];
      if (o.nt == 0) break;
      const int jobs = o.jobs(), G = p.G;
      const int gr = (o.two ? w * o.row_tile : 0) + wl;   // row of the item
      const int rows_here = o.two ? (w ? o.rows - o.row_tile : min(o.rows, o.row_tile)) : o.rows;
      const bool mine = wl < rows_here;
      const bool busy = (wl & ~31) < rows_here;           // this warp has rows
      const int R = o.r0 + gr, t = mine ? R / G : 0;
      const uint64_t nodes = all_nodes(o.n);
      uint64_t mask = 0;
      if (mine) mask = p.mask != nullptr ? p.mask[p.cu_q[o.b] + t] & nodes : all_nodes(t + 1);
      const uint64_t some = KV == kKv16 ? seen_by_lane(p, o.b, o.n) : 0;
      float scale = p.scale_log2;
      if (kScaledQ && mine) scale *= __int_as_float((127 + q_exp[(nth & 1) * kTreeRows + gr]) << 23);
      float m = -INFINITY, l = 0.f;
      for (int j = w; j < jobs; j += 2) {
        const int tile = o.tile_of(j), off = o.L - o.n - (o.tile0 + tile) * kTreeTile;  // columns before the drafted rows
        const bool edge = off < kTreeTile;
        wait(s_full0 + 8 * w, s_phase & 1);
        ++s_phase;
        __syncwarp();
        tc::fence_after_sync();
        if (busy) {
          const bool anew = begins_anew(j, jobs);
          if (kLong && j > 1) {  // the group's earlier products are done: this tile's scores were committed behind them
            const bool last = j + 2 >= jobs, has_sums = j >> 1 > kSumMask + 1;
            if (last ? has_sums : anew) {
              float coef = 0.f;
              if (has_sums) {
                const float2 has = *own_ml;
                coef = has.x == -INFINITY ? 0.f : dev::ex2((has.x - m) * scale);
                l = fmaf(coef, has.y, l);
              }
              move_sums<D>(to, p.sums + (int64_t)(2 * blockIdx.x + w) * D * kTreeTile + 4 * wl, coef, last);
              if (!last) {
                *own_ml = make_float2(m, l);
                l = 0.f;
              }
            }
          }
          weigh<D, Op>(ts, to, edge, mask, off, scale, mine, anew, m, l);
          tc::wait_st();
        }
        if (KV == kKv16 && edge) {
          // V rows that no token sees (behind the sequence, of padding nodes) become 0: a weight of 0 times what they
          // hold could be NaN.
          const uint64_t any = p.mask != nullptr ? seen_by_any(some) : nodes;
          uint32_t gone[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) gone[c] = ~seen(any, off, c);
          if (gone[0] | gone[1] | gone[2] | gone[3]) {
            const uint32_t i = base + o.seq_v(tile), slot = i % nslot;
            wait(op_full0 + 8 * slot, (i / nslot) & 1);
            const int ch = wl % CPR;
            uint8_t* vs = slots + slot * kOperand + (ch >> 3) * kHalf + (ch & 7) * 16;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              for (int row = wl / CPR; row < 32; row += 128 / CPR)
                if (gone[c] >> row & 1) *reinterpret_cast<uint4*>(vs + (32 * c + row) * 128) = make_uint4(0u, 0u, 0u, 0u);
            tc::fence_proxy_async_smem();
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(p_ready0 + 8 * w);
      }

      // The item's end (or this CTA's share of it).
      m = fmaf(m, scale, -weight_exponent<Op>());  // l and O are sums of 2^(score - m) from here on
      const bool both = !o.two && jobs > 1;
      if (!o.two) *own_ml = make_float2(m, l);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (k < jobs) {
          wait(o_full0 + 8 * k, o_phase[k] & 1);
          ++o_phase[k];
        }
      __syncwarp();
      tc::fence_after_sync();
      float c0 = 1.f, c1 = 0.f;
      if (!o.two) {
        // The groups' results of alternate tiles: each takes half the columns of both.
        tc::named_sync(1, 256);
        const float2 a = *reinterpret_cast<const float2*>(ml + 2 * wl), b = *reinterpret_cast<const float2*>(ml + 256 + 2 * wl);
        m = fmaxf(a.x, b.x);
        c0 = a.x == -INFINITY ? 0.f : dev::ex2(a.x - m);
        c1 = b.x == -INFINITY ? 0.f : dev::ex2(b.x - m);
        l = c0 * a.y + c1 * b.y;
      }
      float* rec = p.part + (int64_t)(2 * blockIdx.x + o.slot) * tree_record_floats(D, p.rec_rows);
      const float inv = o.whole ? l > 0.f ? 1.f / l : 0.f : 1.f;
      const uint64_t f0 = pair(c0 * inv, c0 * inv), f1 = pair(c1 * inv, c1 * inv);
      const int64_t out_row = (int64_t)(p.cu_q[o.b] + t) * p.Hq + o.kvh * G + (R - t * G);
      if (mine && (o.two || w == 0)) {
        if (!o.whole) {
          __stcg(rec + gr, m);
          __stcg(rec + p.rec_rows + gr, l);
        } else if (p.lse != nullptr) {
          p.lse[out_row] = l > 0.f ? fmaf(m, dev::kLn2, logf(l)) : l == 0.f ? -INFINITY : l;
        }
      }
      __syncwarp();
      if (busy) {
        // 64 values at a time: one row tile: 32 columns of both groups; two: 64 of the group's own.
        const int col0 = o.two ? 0 : w * (D / 2);
        const uint32_t oc = lanes + kTmemO + (o.two ? w * kTmemS : col0);
#pragma unroll 1
        for (int c = 0; c < D; c += 64) {
          uint32_t y[64];
          uint64_t f[32];
          const int col = col0 + (o.two ? c : c / 2), pairs = o.two ? 32 : 16;
          ld32(oc + (o.two ? c : c / 2), y);
          ld32(oc + (o.two ? c + 32 : c / 2 + kTmemS), y + 32);
          tc::wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k)
            f[k] = mul_pair(pair(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1])), f0);
          if (both) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              f[k] = fma_pair(pair(__uint_as_float(y[2 * k + 32]), __uint_as_float(y[2 * k + 33])), f1, f[k]);
          }
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            if (k >= pairs || !mine) break;
            const float2 a = unpair(f[k]), b = unpair(f[k + 1]), d = unpair(f[k + 2]), e = unpair(f[k + 3]);
            if (o.whole) {
              *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.out) + out_row * D + col + 2 * k) =
                  make_uint4(dev::pack2<T>(a.x, a.y), dev::pack2<T>(b.x, b.y), dev::pack2<T>(d.x, d.y), dev::pack2<T>(e.x, e.y));
            } else {
              // Column by column: the rows of a warp lie together.
              float4* at = reinterpret_cast<float4*>(rec + 2 * p.rec_rows) + (int64_t)((col + 2 * k) / 4) * p.rec_rows + gr;
              __stcg(at, make_float4(a.x, a.y, b.x, b.y));
              __stcg(at + p.rec_rows, make_float4(d.x, d.y, e.x, e.y));
            }
          }
          __syncwarp();
        }
      }
      tc::fence_before_sync();
      wait(q_full0 + 8 * ((nth + 1) & 1), ((nth + 1) >> 1) & 1);  // the next portion is said, its queries are there
      // O and the exchanged sums are read.  All threads of both groups go on, or none (a wait was given up).
      if (tc::named_sync_or(1, 256, *(volatile int*)dead != 0)) break;
      base += 2 * o.nt;
    }
  } else if (warp < kConvertWarp) {
    regs_dec<other_regs(KV)>();
    if (warp == kLoadWarp) {
    // ---------------- loads: a lane issues a box (a page's rows, or half the columns)
    const uint64_t policy = dev::l2_evict_first_policy();
    constexpr int NBOX = KV == kKv16 ? D / 64 : 1;
    constexpr int kUnit = KV == kKvE2m1 ? kBlockTokens : 1;
    constexpr int kLoadBytes = KV == kKv16 ? kOperand : kRaw;
    constexpr int kBoxRow = KV == kKv16 ? 128 : kRaw / kTreeTile;  // bytes of a token's row in a box
    const int pieces = kTreeTile / p.box_rows, boxes = pieces * NBOX;
    const int piece = lane / NBOX, bx = lane - piece * NBOX, r = piece * p.box_rows;
    const bool paged = p.block_table != nullptr;
    // Cache row of a tile, or of this lane's piece of it.
    auto row_of = [&](int t0) {
      if (!paged) return p.base[o.b] + t0;
      // Boxes past the end of the sequence reload its last page; an index outside the pool reads zeros.
      const int pg = min((t0 + r) >> p.page_shift, (o.L - 1) >> p.page_shift);
      const uint32_t page = (uint32_t)p.block_table[(int64_t)o.b * p.bt_stride + pg];
      return page < (uint32_t)p.num_pages ? (int)(page << p.page_shift) + ((t0 + r) & ((1 << p.page_shift) - 1))
                                          : p.num_pages << p.page_shift;
    };
    // The first tiles into L2 while the kernels before still run.  That hands no data over, so it cannot show what they
    // are still writing.  (A page table may itself be on its way.)
    if (!paged && lane < NBOX)
      for (int s = 0; s < min(2 * o.nt, kPrefetch); ++s)
        dev::tma_prefetch_l2_3d(o.is_v(s) ? &p.tm_v : &p.tm_k, bx * 64, o.kvh, row_of((o.tile0 + o.load_tile(s)) * kTreeTile) / kUnit);
    dev::pdl_wait();
    if (p.test_skip_loads && blockIdx.x == 0) more = false;
    const uint32_t ring = dev::smem_addr(KV == kKv16 ? slots : raws);
    Place at;
    at.parity = 1;  // a slot that was never used is free
    for (; more; more = cur.next(p, o)) {
      const int loads = 2 * o.nt, kvh = o.kvh;
      const bool two = o.two;
      int next_t[2] = {o.tile0 * kTreeTile, o.tile0 * kTreeTile};  // of K, of V
      bool v = false;
      for (int s = 0; s < loads; ++s) {
        const int t0 = next_t[v];
        const uint32_t bar = full0 + 8 * at.slot, dst = ring + at.slot * (KV == kKv16 ? kOperand : kRaw);
        const CUtensorMap* map = v ? &p.tm_v : &p.tm_k;
        if (pieces == 1) {
          // One lane: all columns of a tile (of a page, where one holds it).
          if (lane == 0) {
            const int row = row_of(t0) / kUnit;
            wait(empty0 + 8 * at.slot, at.parity);
            if (!*(volatile int*)dead) {
              dev::mbar_arrive_expect_tx(bar, kLoadBytes);
#pragma unroll
              for (int i = 0; i < NBOX; ++i) dev::tma_load_3d(dst + i * kHalf, map, i * 64, kvh, row, bar, policy);
            }
          }
        } else {
          const int row = lane < boxes ? row_of(t0) / kUnit : 0;
          wait(empty0 + 8 * at.slot, at.parity);
          if (!__any_sync(0xffffffffu, *(volatile int*)dead)) {
            if (lane == 0) dev::mbar_arrive_expect_tx(bar, kLoadBytes);
            __syncwarp();
            if (lane < boxes) dev::tma_load_3d(dst + bx * kHalf + r * kBoxRow, map, bx * 64, kvh, row, bar, policy);
          }
        }
        at.advance(1, nload);
        next_t[v] = t0 + kTreeTile;
        // K and V in turn, but of one row tile the second K comes ahead of the first V.
        v = two || s > 0 || loads == 2 ? !v : false;
        if (s == loads - 2) v = true;
      }
    }
    } else if (warp == kMmaWarp) {
    // ---------------- products: the whole warp keeps track, so that addresses are uniform; one lane issues
    constexpr uint32_t kIdS = tc::idesc_f16(kBf16, false, false, kTreeTile, kTreeTile);
    constexpr uint32_t kIdO = tc::idesc_f16(kBf16, false, true, kTreeTile, D);
    const uint32_t q0 = dev::smem_addr(smem), slot0 = dev::smem_addr(slots);
    const bool leader = elect_one();
    // The queries come behind this wait in other warps.  A bounded wait for them that began ahead of it would count the time
    // that the kernels before take, however long, and give the CTA up over a second of it.
    dev::pdl_wait();
    Place first;  // of the portion's loads
    uint32_t p_parity[2] = {0, 0};
    for (uint32_t k = 0;; ++k) {
      wait(q_full0 + 8 * (k & 1), (k >> 1) & 1);
      const Portion o = said[k % 3];
      if (__any_sync(0xffffffffu, o.nt == 0 || *(volatile int*)dead)) break;
      const int jobs = o.jobs();
      tc::fence_after_sync();
      const bool two = o.two;
      const int nt = o.nt;
      Place kp = first, vp = first;
      vp.advance(two || nt == 1 ? 1 : 2, nslot);
      // S of job j, whose K is there: issued by the leader.
      auto scores = [&](int j, uint32_t slot) {
        const int w = j & 1;
        const uint32_t at = ((two ? w * kOperand : 0) + q0), ka = slot0 + slot * kOperand;
        const uint64_t qd = tc::smem_desc(at, 16, 1024, tc::kSwizzle128B), kd = tc::smem_desc(ka, 16, 1024, tc::kSwizzle128B);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_f16_ss(w * kTmemS, qd + (((kk >> 2) * kHalf + (kk & 3) * 32) >> 4), kd + (((kk >> 2) * kHalf + (kk & 3) * 32) >> 4),
                         kIdS, kk > 0);
        tc::commit(s_full0 + 8 * w);
        if (!two || w == 1) tc::commit(op_empty0 + 8 * slot);
        if (j == jobs - 1) tc::commit(q_empty);
      };
      auto next_k = [&](int j) { if (!two || (j & 1)) kp.advance(two || j > 0 ? 2 : 1, nslot); };
      for (int j = 0; j < min(jobs, 2); ++j) {
        if (leader) {
          wait(op_full0 + 8 * kp.slot, kp.parity);
          tc::fence_after_sync();
          scores(j, kp.slot);
        }
        next_k(j);
      }
      for (int j = 0; j < jobs; ++j) {
        const int w = j & 1;
        const uint32_t slot = vp.slot;
        const bool again = j + 2 < jobs;
        if (leader) {
          wait(op_full0 + 8 * slot, vp.parity);
          wait(p_ready0 + 8 * w, p_parity[w]);
          tc::fence_after_sync();
          const uint64_t vd = tc::smem_desc(slot0 + slot * kOperand, kHalf, 1024, tc::kSwizzle128B);
          const uint32_t ps = w * kTmemS, od = kTmemO + w * kTmemS;
#pragma unroll
          for (int kk = 0; kk < kTreeTile / 16; ++kk) {
            mma_f16_ts(od, ps + (kk >> 1) * 32 + (kk & 1) * 8, vd + (kk * 2048 >> 4), kIdO, !begins_anew(j, jobs) || kk > 0);
            if (kBf16) mma_f16_ts(od, ps + (kk >> 1) * 32 + (kk & 1) * 8 + 16, vd + (kk * 2048 >> 4), kIdO, 1u);
          }
          if (!two || w == 1) tc::commit(op_empty0 + 8 * slot);
          if (!again) {
            tc::commit(o_full0 + 8 * w);
          } else {
            wait(op_full0 + 8 * kp.slot, kp.parity);
            tc::fence_after_sync();
            scores(j + 2, kp.slot);
          }
        }
        if (again) next_k(j + 2);
        p_parity[w] ^= 1;
        // The last V, of one row tile, follows the one before it; behind it begins the next portion.
        const int left = nt - 1 - (two ? j >> 1 : j);
        if (!two || w == 1) vp.advance(left == 0 || (left == 1 && !two) ? 1 : 2, nslot);
      }
      first = vp;
    }
    } else {
    // ---------------- queries of the items behind the first
    // Portion k is said and its queries are written once portion k - 1's products with Q are done; the softmax groups
    // wait for that at the end of k - 1, so neither of the two barriers nor the three places are ever overrun.
    put_queries(o, tid - 64, 256 + 32 * kQueryWarps, -1);
    tc::named_sync(2, 256 + 32 * kQueryWarps);
    if (lane == 0) dev::mbar_arrive(q_full0);
    for (uint32_t k = 1; more; ++k) {
      more = cur.next(p, o);
      if (more) put_queries(o, tid - 32 * kQueryWarp, 32 * kQueryWarps, (int)k - 1);
      else wait(q_empty, (k - 1) & 1);
      if (!more) o.nt = 0;
      if (warp == kQueryWarp && lane == 0) said[k % 3] = o;
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(q_full0 + 8 * (k & 1));
    }
    }
  } else {
    if constexpr (KV != kKv16) regs_dec<kConvertRegs>();
    // ---------------- widening of 8- and 4-bit rows
    if constexpr (KV != kKv16) {
      // Two teams of two warps take alternate operands.  A step takes 64 chunks twice over, as 128 threads would: from
      // one to the next a chunk's row within 8 and its place in the row stay, a constant offset on both sides.
      const int team = (warp - kConvertWarp) >> 1;
      constexpr int kSteps = kTreeTile * CPR / 128, kBatch = 8;
      constexpr int kBlock = kRaw / 8;                    // bytes of a 4-bit block in the ring
      // K (and E4M3): neighbouring lanes along a row; V of 4 bits: along the tokens, whose codes lie together.
      int krow[2], kch, vrow, vch[2], k_to[2], v_to[2], v_from[2];
      kch = (tid & 63) % CPR;
      vrow = tid & 15;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int ct = (tid & 63) + 64 * v;
        krow[v] = ct / CPR;
        vch[v] = ct >> 4;
        k_to[v] = (kch >> 3) * kHalf + krow[v] * 128 + (((kch & 7) ^ (krow[v] & 7)) << 4);
        v_to[v] = vrow * 128 + (((vch[v] & 7) ^ (vrow & 7)) << 4);
        const int g = 8 * vch[v] / (D / 8), swap = ((D == 128 ? g : g >> 1) & 1) << 2;
        v_from[v] = g * D + ((vrow >> 1) ^ swap) * (D / 8) + (vrow & 1) * (D / 16) + (8 * vch[v] % (D / 8)) / 2;
      }
      Place raw, op;
      raw.slot = op.slot = team;
      dev::pdl_wait();
      for (; more; more = cur.next(p, o)) {
        const uint64_t some = seen_by_lane(p, o.b, o.n);
        for (int s = team; s < 2 * o.nt; s += 2) {
          const bool is_v = o.is_v(s);
          wait(full0 + 8 * raw.slot, raw.parity);
          wait(op_empty0 + 8 * op.slot, op.parity ^ 1);
          const uint8_t* src = raws + raw.slot * kRaw;
          uint8_t* dst = slots + op.slot * kOperand;
          if constexpr (KV == kKvE4m3) {
#pragma unroll
            for (int i0 = 0; i0 < kSteps; i0 += kBatch) {
              uint2 x[2 * kBatch];
#pragma unroll
              for (int i = 0; i < 2 * kBatch; ++i)
                x[i] = *reinterpret_cast<const uint2*>(src + 8 * (tid & 63) + (i & 1) * 512 + (i0 + i / 2) * 1024);
#pragma unroll
              for (int i = 0; i < 2 * kBatch; ++i) {
                uint4 y;
                dev::e4m3x4_to_f16x4(x[i].x, y.x, y.y);
                dev::e4m3x4_to_f16x4(x[i].y, y.z, y.w);
                *reinterpret_cast<uint4*>(dst + k_to[i & 1] + (i0 + i / 2) * (128 / CPR) * 128) = y;
              }
            }
          } else {
            // Eight elements of one scale.
            auto widen = [&](uint32_t codes, uint32_t scale) {
              const uint32_t z = dev::e4m3x2_to_f16x2(scale), s2 = __byte_perm(z, z, 0x1010);
              uint32_t f[4];
              dev::e2m1x8_to_f16x8(codes, f);
              return make_uint4(dev::hmul2(f[0], s2), dev::hmul2(f[1], s2), dev::hmul2(f[2], s2), dev::hmul2(f[3], s2));
            };
            // A step goes 128 / CPR rows on (K), or 128 / CPR / 16 blocks, or half a row of them (V).
            constexpr int kHalves = D / 64;               // steps per block
#pragma unroll
            for (int i0 = 0; i0 < kSteps; i0 += kBatch) {
              uint32_t x[2 * kBatch], z[2 * kBatch];
#pragma unroll
              for (int i = 0; i < 2 * kBatch; ++i) {
                const int v = i & 1, blk = (i0 + i / 2) / kHalves, half = (i0 + i / 2) % kHalves;
                const uint8_t* at = src + blk * kBlock;
                if (is_v) {
                  x[i] = *reinterpret_cast<const uint32_t*>(at + v_from[v] + half * 4 * D);
                  z[i] = at[8 * D + 16 * (vch[v] >> 1) + vrow + half * 64];
                } else {
                  x[i] = *reinterpret_cast<const uint32_t*>(at + krow[v] * (D / 2) + 4 * kch + half * 4 * D);
                  z[i] = at[8 * D + krow[v] * (D / 16) + (kch >> 1) + half * (D / 2)];
                }
              }
#pragma unroll
              for (int i = 0; i < 2 * kBatch; ++i) {
                const int v = i & 1, blk = (i0 + i / 2) / kHalves, half = (i0 + i / 2) % kHalves;
                *reinterpret_cast<uint4*>(dst + blk * 2048 + (is_v ? v_to[v] + half * kHalf : k_to[v] + half * 1024)) = widen(x[i], z[i]);
              }
            }
          }
          const int off = o.L - o.n - (o.tile0 + o.load_tile(s)) * kTreeTile;
          if (is_v && off < kTreeTile) {
            // V rows that no token sees become 0.
            const uint64_t any = seen_by_any(some);
            uint32_t gone[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) gone[c] = ~seen(any, off, c);
            if (gone[0] | gone[1] | gone[2] | gone[3]) {
              tc::named_sync(3 + team, 64);
#pragma unroll
              for (int c = 0; c < 4; ++c)
                for (int row = krow[0]; row < 32; row += 64 / CPR)
                  if (gone[c] >> row & 1)
                    *reinterpret_cast<uint4*>(dst + (kch >> 3) * kHalf + (32 * c + row) * 128 + (kch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            dev::mbar_arrive(op_full0 + 8 * op.slot);
            dev::mbar_arrive(empty0 + 8 * raw.slot);
          }
          raw.advance(2, nraw);
          op.advance(2, nslot);
        }
      }
    }
  }
  __syncthreads();
  if (*(volatile int*)dead) {
    // Given up: copies and products may be in flight.  They need far less than this to end.
    const uint64_t start = dev::global_timer_ns();
    while (dev::global_timer_ns() - start < 20000000ull) {}
    __syncthreads();
    if (warp < kMmaWarp) leave_nan<D>(p);
  }
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(0, kTmemAll);
  }
}

// ------------------------------------------------------------------ combination

// 32 query rows (lanes) of one item that several CTAs share: a warp takes an eighth of the columns and every GROUPS-th
// record, then the groups meet in shared memory.  Bound by the latency of the records' loads from L2: more groups where
// records are many or blocks few.  (Always 8: 64 heads x 64 drafts over 32K tokens 81.6 us instead of 80.7; always 2: 4K
// tokens, with 19 records an item, 18.9 us instead of 11.4.)
FD_HD constexpr int combine_parts(int groups) { return groups == 2 ? 8 : groups == 4 ? 4 : 1; }  // eighths of a block
template <typename T, int D, int GROUPS>
__global__ void __launch_bounds__(32 * GROUPS * combine_parts(GROUPS)) fd_tree_combine_kernel(const __grid_constant__ TreeParams p) {
  constexpr int NQ = D / 32, PARTS = combine_parts(GROUPS);  // NQ: groups of four columns of a warp
  __shared__ float sm_m[GROUPS - 1][PARTS][32], sm_l[GROUPS - 1][PARTS][32];
  __shared__ float4 sm_o[GROUPS - 1][PARTS][NQ][32];
  dev::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, place = warp % PARTS, group = warp / PARTS;
  const int cta = p.split[blockIdx.y], rb = blockIdx.x, part = blockIdx.z * PARTS + place, col = part * (D / 8);
  // The item that CTA `cta` goes on with; CTA cta - 1 began it.
  const int u = tree_run_begin(p, cta);
  int b = 0, hi = p.B;
  while (hi - b > 1) {
    const int mid = (b + hi) >> 1;
    if (p.unit_base[mid] <= u) b = mid; else hi = mid;
  }
  const int n = p.cu_q[b + 1] - p.cu_q[b], all = n * p.G, groups = tree_groups(all);
  const int per = tree_item_units(p, tree_tiles(p.len[b])), item = (u - p.unit_base[b]) / per;
  const int end = p.unit_base[b] + (item + 1) * per;
  const int kvh = item / groups, r0 = (item - kvh * groups) * kTreeRows, rows = min(all - r0, kTreeRows);
  const int gr = rb * 32 + lane;
  if (rb * 32 >= rows) return;
  int records = 1;
  while (cta + records - 1 < p.ctas && tree_run_begin(p, cta + records - 1) < end) ++records;
  const int64_t size = tree_record_floats(D, p.rec_rows);
  auto record = [&](int i) { return p.part + (int64_t)(2 * (cta - 1 + i) + (i == 0)) * size; };
  dev::pdl_wait();
  float m = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int i = group; i < records; i += GROUPS) m = fmaxf(m, __ldcg(record(i) + gr));
  float4 acc[NQ];
#pragma unroll
  for (int k = 0; k < NQ; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = group; i < records; i += GROUPS) {
    const float* rec = record(i);
    const float mi = __ldcg(rec + gr), li = __ldcg(rec + p.rec_rows + gr);
    const float c = mi == -INFINITY ? 0.f : dev::ex2(mi - m);
    l = fmaf(c, li, l);
#pragma unroll
    for (int k = 0; k < NQ; ++k) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(rec + 2 * p.rec_rows) + (int64_t)(col / 4 + k) * p.rec_rows + gr);
      acc[k].x = fmaf(c, x.x, acc[k].x);
      acc[k].y = fmaf(c, x.y, acc[k].y);
      acc[k].z = fmaf(c, x.z, acc[k].z);
      acc[k].w = fmaf(c, x.w, acc[k].w);
    }
  }
  if (group > 0) {
    sm_m[group - 1][place][lane] = m;
    sm_l[group - 1][place][lane] = l;
#pragma unroll
    for (int k = 0; k < NQ; ++k) sm_o[group - 1][place][k][lane] = acc[k];
  }
  __syncthreads();
  if (group > 0 || gr >= rows) return;
  float top = m;
#pragma unroll
  for (int g = 0; g < GROUPS - 1; ++g) top = fmaxf(top, sm_m[g][place][lane]);
  const float c0 = m == -INFINITY ? 0.f : dev::ex2(m - top);
  l *= c0;
#pragma unroll
  for (int k = 0; k < NQ; ++k) acc[k] = make_float4(acc[k].x * c0, acc[k].y * c0, acc[k].z * c0, acc[k].w * c0);
#pragma unroll
  for (int g = 0; g < GROUPS - 1; ++g) {
    const float mg = sm_m[g][place][lane], c = mg == -INFINITY ? 0.f : dev::ex2(mg - top);
    l = fmaf(c, sm_l[g][place][lane], l);
#pragma unroll
    for (int k = 0; k < NQ; ++k) {
      const float4 x = sm_o[g][place][k][lane];
      acc[k].x = fmaf(c, x.x, acc[k].x);
      acc[k].y = fmaf(c, x.y, acc[k].y);
      acc[k].z = fmaf(c, x.z, acc[k].z);
      acc[k].w = fmaf(c, x.w, acc[k].w);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int R = r0 + gr, t = R / p.G;
  const int64_t out_row = (int64_t)(p.cu_q[b] + t) * p.Hq + kvh * p.G + (R - t * p.G);
#pragma unroll
  for (int k = 0; k < NQ; k += 2)
    *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.out) + out_row * D + col + 4 * k) =
        make_uint4(dev::pack2<T>(acc[k].x * inv, acc[k].y * inv), dev::pack2<T>(acc[k].z * inv, acc[k].w * inv),
                   dev::pack2<T>(acc[k + 1].x * inv, acc[k + 1].y * inv), dev::pack2<T>(acc[k + 1].z * inv, acc[k + 1].w * inv));
  if (part == 0 && p.lse != nullptr) p.lse[out_row] = l > 0.f ? fmaf(top, dev::kLn2, logf(l)) : l == 0.f ? -INFINITY : l;
}

// ------------------------------------------------------------------ launch

template <typename T, int D, int KV>
cudaError_t launch(const TreeParams& p, int splits, cudaStream_t stream) {
  const bool is_long = p.sums != nullptr;
  const void* fn = is_long ? reinterpret_cast<const void*>(&fd_tree_kernel<T, D, KV, true>)
                           : reinterpret_cast<const void*>(&fd_tree_kernel<T, D, KV, false>);
  int dev_id = 0;
  cudaError_t err = cudaGetDevice(&dev_id);
  if (err != cudaSuccess) return err;
  static uint64_t done_masks[2] = {0, 0};  // devices whose shared-memory limit is set for these kernels
  uint64_t* const done_mask = &done_masks[is_long];
  const uint64_t bit = 1ull << (dev_id & 63);
  if (!(__atomic_load_n(done_mask, __ATOMIC_ACQUIRE) & bit)) {
    err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kTreeSmemBytes);
    if (err != cudaSuccess) return err;
    __atomic_fetch_or(done_mask, bit, __ATOMIC_RELEASE);
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(threads(KV));
  cfg.dynamicSmemBytes = kTreeSmemBytes;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void* args[] = {const_cast<TreeParams*>(&p)};
  err = cudaLaunchKernelExC(&cfg, fn, args);
  if (err != cudaSuccess || splits == 0) return err;
  const int blocks = p.rec_rows / 32 * splits;
  const int groups = p.ctas / splits < 3 ? 2 : blocks >= 128 ? 4 : 8;  // ctas / splits + 1: records of an item
  cfg.gridDim = dim3(p.rec_rows / 32, splits, 8 / combine_parts(groups));
  cfg.blockDim = dim3(32 * groups * combine_parts(groups));
  cfg.dynamicSmemBytes = 0;
  const void* combine = groups == 2   ? reinterpret_cast<const void*>(&fd_tree_combine_kernel<T, D, 2>)
                        : groups == 4 ? reinterpret_cast<const void*>(&fd_tree_combine_kernel<T, D, 4>)
                                      : reinterpret_cast<const void*>(&fd_tree_combine_kernel<T, D, 8>);
  return cudaLaunchKernelExC(&cfg, combine, args);
}

}  // namespace tree
}  // namespace fd
