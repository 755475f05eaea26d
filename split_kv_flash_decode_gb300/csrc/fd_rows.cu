// Cache rows: fd_append (norm, rotation and store of new tokens) and fd_gather (rows of a
// cache back in 16 bits).  See fd.h for the contract.
//
// Both are bound by the bytes they move.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <new>

#include "fd_host.h"
#include "fd_kernel.cuh"

struct fd_rows_s {
  int B, Hq, Hkv, d, dtype, page_size, max_pages;
  int64_t T, cache_bytes;
  int32_t cu[FD_MAX_BATCH + 1];   // prefix sums of count
  int32_t begin[FD_MAX_BATCH];    // row in its sequence of the first token
  int32_t base[FD_MAX_BATCH];     // contiguous caches: cache row of the sequence's row 0
};

namespace fd {
namespace {

constexpr int kRowsThreads = 128;
constexpr int kMaxAxes = 4;
constexpr int kMaxPairs = 64;
constexpr double kMaxFreq = 1 << 20;
// Warps that an append is split into while it has enough head rows: 16 on each of 152 SMs.  (2090
// tokens of 40 head rows: 11.5 us with 16; 32 and 64 took 1.2 and 2.1 us more: a token's angles are computed
// once per warp.)
constexpr int64_t kAppendWarps = 16 * 152;

// Tokens of one gather warp: two rounds of its lanes.  (32K tokens of a 4-bit cache, 172 MB: 27.2 us;
// with one round 34.0, three 27.6, four 28.5 us.)
FD_HD constexpr int gather_tokens(int d) { return 2 * (512 / d); }

// Where the rows of a call lie.
struct RowMap {
  int32_t B, Hkv, page_shift, num_pages, bt_stride;
  const int32_t* block_table;  // nullptr: contiguous
  uint32_t* status;
  int32_t cu[FD_MAX_BATCH + 1];
  int32_t begin[FD_MAX_BATCH];
  int32_t base[FD_MAX_BATCH];
};

struct AppendParams {
  RowMap m;
  const void *q, *k, *v, *q_weight, *k_weight;
  int64_t q_stride[2], k_stride[2], v_stride[2];
  void *q_out, *k_out, *k_cache, *v_cache;
  const int32_t* positions;
  int64_t pos_stride;
  float eps, weight_offset, k_mul, v_mul, rope_scale;
  int32_t T, Hq, q_norm, k_norm, rot, interleaved;
  int32_t rows_per_warp, splits;   // head rows of one warp; warps per token
  uint64_t freq[kMaxPairs];        // turns per position, in units of 2^-64
  uint8_t axis[kMaxPairs];
};
static_assert(sizeof(AppendParams) <= 4096, "kernel parameters must stay within 4 KB");

struct GatherParams {
  RowMap m;
  const void *k_cache, *v_cache;
  void *k_out, *v_out;
  int32_t T;
};

// Sequence of token t: the last b with cu[b] <= t (sequences without tokens are skipped).
__device__ __forceinline__ int find_sequence(const RowMap& m, int t) {
  int lo = 0, hi = m.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (m.cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Cache row (token units) of row r of sequence b, or -1 when its page is outside the pool.
__device__ __forceinline__ int64_t cache_row(const RowMap& m, int b, int r) {
  if (m.block_table == nullptr) return (int64_t)m.base[b] + r;
  const int pg = m.block_table[(int64_t)b * m.bt_stride + (r >> m.page_shift)];
  if ((uint32_t)pg >= (uint32_t)m.num_pages) {
    if (m.status != nullptr) atomicOr(m.status, 1u);
    return -1;
  }
  return ((int64_t)pg << m.page_shift) + (r & ((1 << m.page_shift) - 1));
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Eight values rounded to E4M3 or E2M1 (saturating), first value in the low bits.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ uint2 to_e4m3x8(const float (&x)[8]) {
  return make_uint2(to_e4m3x4(x[0], x[1], x[2], x[3]), to_e4m3x4(x[4], x[5], x[6], x[7]));
}
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// The E4M3 scale of a block of 16 elements, 8 of them in each of two neighbouring lanes, and the
// codes of this lane's 8.  The quotient is a true division: with the product by a reciprocal,
// values half-way between two codes (common: 16-bit values over a scale of 4 significant bits)
// would not always round to even.
__device__ __forceinline__ void quantise(const float (&y)[8], uint32_t& scale, uint32_t& codes) {
  float m = fabsf(y[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(y[i]));
  m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
  scale = to_e4m3x4(m / 6.f, 0.f, 0.f, 0.f) & 0xffu;
  const float s = dev::Elem<__half>::to_f2(dev::e4m3x2_to_f16x2(scale)).x;
  const bool any = s > 0.f;  // false for a NaN scale too: the codes do not matter then
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = any ? y[i] / s : 0.f;
  codes = to_e2m1x8(z);
}

// Byte offset in a 4-bit V block of element e (a multiple of 8) of row r.
template <int D>
__device__ __forceinline__ int v_offset(int r, int e) {
  const int g = e / (D / 8), swap = ((D == 128 ? g : g >> 1) & 1) << 2;
  return g * D + (((r >> 1) ^ swap) * (D / 8)) + (r & 1) * (D / 16) + (e % (D / 8)) / 2;
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(dev::pack2<T>(f[0], f[1]), dev::pack2<T>(f[2], f[3]), dev::pack2<T>(f[4], f[5]),
                    dev::pack2<T>(f[6], f[7]));
}

// A head row of D elements takes D / 16 lanes.  A lane has two runs of 8 elements: the two halves
// of its rotation pairs (below rot), or plain runs (above), so that a pair never leaves its lane
// and every load and store is 16 bytes wide.  One warp: one token, rows_per_warp of its Hq + 2 Hkv
// head rows (q, then k, then v), 512 / D of them at a time.  The angles depend on the token alone:
// each lane computes 8 / (512 / D) of the eight it needs, the lanes of the warp's other rows the
// rest.  Position x frequency is a 64-bit product of turns that wraps where whole turns drop out,
// so no position is too far.
//
// Bound by HBM: 805 MB (32K tokens of 48 head rows) in 126 us, 6.4 TB/s; fewer tokens by the chain of
// each warp's rows, so two rounds of rows are on their way ahead of the one at work (2090 tokens of 40
// head rows: 11.5 us; with one round ahead 12.1).  Many warps keep the loads in flight: 7 blocks per
// SM (72 registers, and 16 bytes a thread that 16-bit caches spill) take 126 us for the 32K tokens,
// 6 take 131, 5 take 140 and 8, which spill more, 129;
// 4-bit caches, whose quantisation needs the registers, are faster with 4.
template <typename T, int D, int KV>
__global__ void __launch_bounds__(kRowsThreads, KV == kKvE2m1 ? 4 : 7) fd_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LPH = D / 16;       // lanes per head row
  constexpr int HPW = 32 / LPH;     // head rows a warp handles at a time
  constexpr int OWN = 8 / HPW;      // angles a lane computes
  dev::pdl_launch_dependents();
  dev::pdl_wait();
  const int64_t wid = (int64_t)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)(wid / p.splits), split = (int)(wid - (int64_t)t * p.splits);
  if (t >= p.T) return;
  const int lane = threadIdx.x & 31, l = lane & (LPH - 1), sub = lane / LPH;
  const int b = find_sequence(p.m, t);
  const int r = p.m.begin[b] + (t - p.m.cu[b]);
  const int64_t row = p.k_cache != nullptr ? cache_row(p.m, b, r) : -1;

  const int Hq = p.q != nullptr ? p.Hq : 0, Hk = p.k != nullptr ? p.m.Hkv : 0;
  const int Hv = p.v != nullptr ? p.m.Hkv : 0;
  const int lo = split * p.rows_per_warp, hi = min(lo + p.rows_per_warp, Hq + Hk + Hv);

  const int half = p.rot >> 1, rl = p.rot >> 4;
  const bool rotates = l < rl;
  const int ea = rotates ? 8 * l : p.rot + 8 * (l - rl);
  const int eb = rotates ? half + 8 * l : ((p.rot + D) >> 1) + 8 * (l - rl);
  // The warp's first rows, on their way while the angles are computed; m: those after them.
  const int first_kind = lo < Hq ? 0 : lo < Hq + Hk ? 1 : 2;
  uint4 na, nb, ma, mb;
  auto load = [&](uint4& na, uint4& nb, const T* src, int64_t stride, int h, int last) {
    const T* at = src + (int64_t)min(h + sub, last - 1) * stride;  // rows past the end repeat the last one
    na = *reinterpret_cast<const uint4*>(at + ea);
    nb = *reinterpret_cast<const uint4*>(at + eb);
  };
  {
    const int64_t* stride = first_kind == 0 ? p.q_stride : first_kind == 1 ? p.k_stride : p.v_stride;
    const void* in = first_kind == 0 ? p.q : first_kind == 1 ? p.k : p.v;
    const int before = first_kind == 0 ? 0 : first_kind == 1 ? Hq : Hq + Hk;
    const T* src = reinterpret_cast<const T*>(in) + (int64_t)t * stride[0];
    const int last = min(hi - before, first_kind == 0 ? Hq : p.m.Hkv);
    load(na, nb, src, stride[1], lo - before, last);
    load(ma, mb, src, stride[1], lo - before + HPW, last);
  }
  // Pair i of a lane: (ea + i, eb + i), or, interleaved, neighbours of run a (i < 4) or run b.
  float c[8], s[8];
  if (p.rot > 0 && lo < Hq + Hk) {
    float co[OWN], so[OWN];
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      const int i = sub * OWN + k;
      co[k] = 1.f;
      so[k] = 0.f;
      if (rotates) {
        const int pair = p.interleaved ? (i < 4 ? 4 * l : (half >> 1) + 4 * l - 4) + i : 8 * l + i;
        const int pos = p.positions != nullptr ? p.positions[p.axis[pair] * p.pos_stride + t] : r;
        const uint64_t turns = (uint64_t)(int64_t)pos * p.freq[pair];
        sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &so[k], &co[k]);
        co[k] *= p.rope_scale;
        so[k] *= p.rope_scale;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = __shfl_sync(0xffffffffu, co[i % OWN], i / OWN * LPH + l);
      s[i] = __shfl_sync(0xffffffffu, so[i % OWN], i / OWN * LPH + l);
    }
  }

  // Rows [first, last) of one kind, `out` in the q type, `kind` 0: q, 1: k, 2: v.
  auto rows = [&](int kind, int first, int last, const void* in, const int64_t* stride,
                  const void* weight, int norm, void* out, int H, void* cache, float mul) {
    if (first >= last) return;
    const T* src = reinterpret_cast<const T*>(in) + (int64_t)t * stride[0];
    const uint4* wa = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(weight) + ea);
    const uint4* wb = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(weight) + eb);
    if (kind != first_kind) {
      load(na, nb, src, stride[1], first, last);
      load(ma, mb, src, stride[1], first + HPW, last);
    }
#pragma unroll 1
    for (int h0 = first; h0 < last; h0 += HPW) {
      {
        const int h = h0 + sub;
        const bool there = h < last;
        float a[8], x[8];
        dev::unpack8<T>(na, a);
        dev::unpack8<T>(nb, x);
        na = ma;
        nb = mb;
        if (h0 + 2 * HPW < last) load(ma, mb, src, stride[1], h0 + 2 * HPW, last);
        if (kind < 2 && norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(x[i], x[i], ss));
#pragma unroll
          for (int off = 1; off < LPH; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          const float n = rsqrtf(ss * (1.f / D) + p.eps);
          if (weight != nullptr) {
            float w[8];
            dev::unpack8<T>(*wa, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = a[i] * n * (w[i] + p.weight_offset);
            dev::unpack8<T>(*wb, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * n * (w[i] + p.weight_offset);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              a[i] *= n;
              x[i] *= n;
            }
          }
        }
        if (kind < 2 && rotates) {
          if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a0 = a[2 * i], x0 = x[2 * i];
              a[2 * i] = a0 * c[i] - a[2 * i + 1] * s[i];
              a[2 * i + 1] = a0 * s[i] + a[2 * i + 1] * c[i];
              x[2 * i] = x0 * c[4 + i] - x[2 * i + 1] * s[4 + i];
              x[2 * i + 1] = x0 * s[4 + i] + x[2 * i + 1] * c[4 + i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a0 = a[i];
              a[i] = a0 * c[i] - x[i] * s[i];
              x[i] = a0 * s[i] + x[i] * c[i];
            }
          }
        }
        if (out != nullptr && there) {
          T* dst = reinterpret_cast<T*>(out) + ((int64_t)t * H + h) * D;
          *reinterpret_cast<uint4*>(dst + ea) = pack8<T>(a);
          *reinterpret_cast<uint4*>(dst + eb) = pack8<T>(x);
        }
        if (kind == 0 || cache == nullptr) continue;
        const bool store = there && row >= 0;
        if constexpr (KV == kKv16) {
          if (store) {
            T* dst = reinterpret_cast<T*>(cache) + (row * H + h) * D;
            *reinterpret_cast<uint4*>(dst + ea) = pack8<T>(a);
            *reinterpret_cast<uint4*>(dst + eb) = pack8<T>(x);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) { a[i] *= mul; x[i] *= mul; }
          if constexpr (KV == kKvE4m3) {
            if (store) {
              uint8_t* dst = reinterpret_cast<uint8_t*>(cache) + (row * H + h) * D;
              *reinterpret_cast<uint2*>(dst + ea) = to_e4m3x8(a);
              *reinterpret_cast<uint2*>(dst + eb) = to_e4m3x8(x);
            }
          } else {
            // The runs of two neighbouring lanes are whole blocks of 16 (rot is a multiple of 32).
            uint32_t sa, sb, ca, cb;
            quantise(a, sa, ca);
            quantise(x, sb, cb);
            if (store) {
              uint8_t* blk = reinterpret_cast<uint8_t*>(cache) + ((row >> kBlockShift) * H + h) * (9 * D);
              const int r16 = (int)(row & (kBlockTokens - 1));
              *reinterpret_cast<uint32_t*>(blk + (kind == 1 ? r16 * (D / 2) + ea / 2 : v_offset<D>(r16, ea))) = ca;
              *reinterpret_cast<uint32_t*>(blk + (kind == 1 ? r16 * (D / 2) + eb / 2 : v_offset<D>(r16, eb))) = cb;
              if ((l & 1) == 0) {
                const int ja = ea / 16, jb = eb / 16;
                blk[8 * D + (kind == 1 ? r16 * (D / 16) + ja : 16 * ja + r16)] = (uint8_t)sa;
                blk[8 * D + (kind == 1 ? r16 * (D / 16) + jb : 16 * jb + r16)] = (uint8_t)sb;
              }
            }
          }
        }
      }
    }
  };
  rows(0, lo, min(hi, Hq), p.q, p.q_stride, p.q_weight, p.q_norm, p.q_out, p.Hq, nullptr, 1.f);
  rows(1, max(lo - Hq, 0), min(hi - Hq, Hk), p.k, p.k_stride, p.k_weight, p.k_norm, p.k_out, p.m.Hkv,
       p.k_cache, p.k_mul);
  rows(2, max(lo - Hq - Hk, 0), min(hi - Hq - Hk, Hv), p.v, p.v_stride, nullptr, 0, nullptr, p.m.Hkv,
       p.v_cache, p.v_mul);
}

// One warp: gather_tokens(D) tokens of one KV head, K (even warps of the grid) or V.  A row takes
// D / 16 lanes, a lane the 8 elements at 8 l and those at D / 2 + 8 l.  Bound by HBM: 172 MB at 6.3
// TB/s (32K tokens from 4 bits), 35 MB in 5.7 us (from E4M3).  Many small warps: each finds its rows
// (a chain of a binary search and a page-table load) while others load.
template <typename T, int D, int KV>
__global__ void __launch_bounds__(kRowsThreads) fd_gather_kernel(const __grid_constant__ GatherParams p) {
  constexpr int LPH = D / 16, HPW = 32 / LPH, TOK = gather_tokens(D);
  dev::pdl_launch_dependents();
  dev::pdl_wait();
  const int64_t wid = (int64_t)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5);
  const int H = p.m.Hkv;
  const int64_t tile = wid / (2 * H);
  const int w = (int)(wid - tile * (2 * H)), h = w >> 1, is_v = w & 1;
  const int64_t t0 = tile * TOK;
  if (t0 >= p.T) return;
  const int lane = threadIdx.x & 31, l = lane & (LPH - 1), sub = lane / LPH;
  // Lane i finds the cache row of token t0 + i.
  int64_t my_row = -1;
  if (lane < TOK && t0 + lane < p.T) {
    const int t = (int)(t0 + lane), b = find_sequence(p.m, t);
    my_row = cache_row(p.m, b, p.m.begin[b] + (t - p.m.cu[b]));
  }
  const int n = (int)min((int64_t)TOK, p.T - t0);
  const uint8_t* cache = reinterpret_cast<const uint8_t*>(is_v ? p.v_cache : p.k_cache);
  T* out = reinterpret_cast<T*>(is_v ? p.v_out : p.k_out) + (t0 * H + h) * D + 8 * l;
#pragma unroll
  for (int i = 0; i < TOK / HPW; ++i) {
    const int tok = i * HPW + sub;
    const int64_t row = __shfl_sync(0xffffffffu, my_row, tok);
    if (tok >= n) continue;
    uint4 y[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (row >= 0) {
      const uint8_t* blk = cache + (KV == kKv16     ? (row * H + h) * (2 * D)
                                    : KV == kKvE4m3 ? (row * H + h) * D
                                                    : ((row >> kBlockShift) * H + h) * (9 * D));
      const int r16 = (int)row & (kBlockTokens - 1);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int e = k * (D / 2) + 8 * l;
        if constexpr (KV == kKv16) {
          y[k] = *reinterpret_cast<const uint4*>(blk + 2 * e);
        } else if constexpr (KV == kKvE4m3) {
          const uint2 x = *reinterpret_cast<const uint2*>(blk + e);
          dev::e4m3x4_to_f16x4(x.x, y[k].x, y[k].y);
          dev::e4m3x4_to_f16x4(x.y, y[k].z, y[k].w);
        } else {
          const uint32_t x = *reinterpret_cast<const uint32_t*>(blk + (is_v ? v_offset<D>(r16, e) : r16 * (D / 2) + e / 2));
          const uint32_t z = dev::e4m3x2_to_f16x2(blk[8 * D + (is_v ? 16 * (e / 16) + r16 : r16 * (D / 16) + e / 16)]);
          const uint32_t s2 = __byte_perm(z, z, 0x1010);
          uint32_t f[4];
          dev::e2m1x8_to_f16x8(x, f);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[j] = dev::hmul2(f[j], s2);
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
              const float2 v = dev::Elem<__half>::to_f2(f[j]);
              f[j] = dev::pack2<T>(v.x, v.y);
            }
          }
          y[k] = make_uint4(f[0], f[1], f[2], f[3]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) *reinterpret_cast<uint4*>(out + (int64_t)tok * H * D + k * (D / 2)) = y[k];
  }
}

int64_t row_bytes(const fd_rows_s* r) { return cache_row_bytes(r->dtype, r->d); }

// Page-table checks shared by both calls, and the map of the rows.
int make_map(const fd_rows_s* r, int num_pages, const int32_t* block_table, int bt_stride,
             uint32_t* status, RowMap* m) {
  m->page_shift = 0;
  if (r->page_size) {
    if (num_pages < 1 || block_table == nullptr || bt_stride < r->max_pages) return FD_ERR_INVALID;
    if ((int64_t)num_pages * r->page_size >= (int64_t)1 << 31) return FD_ERR_UNSUPPORTED;
    while ((1 << m->page_shift) < r->page_size) ++m->page_shift;
  } else if (block_table != nullptr) {
    return FD_ERR_INVALID;
  }
  if (!aligned(block_table, 4) || !aligned(status, 4)) return FD_ERR_ALIGN;
  m->B = r->B;
  m->Hkv = r->Hkv;
  m->num_pages = num_pages;
  m->bt_stride = bt_stride;
  m->block_table = block_table;
  m->status = status;
  std::memcpy(m->cu, r->cu, sizeof(m->cu));
  std::memcpy(m->begin, r->begin, sizeof(m->begin));
  std::memcpy(m->base, r->base, sizeof(m->base));
  return FD_OK;
}

int launch_rows(const void* fn, int64_t warps, void* params, cudaStream_t stream) {
  const int64_t blocks = (warps + kRowsThreads / 32 - 1) / (kRowsThreads / 32);
  if (blocks >= (int64_t)1 << 31) return FD_ERR_UNSUPPORTED;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kRowsThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void* args[] = {params};
  if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) {
    cudaGetLastError();
    return FD_ERR_CUDA;
  }
  return FD_OK;
}

template <template <typename, int, int> class K>
const void* pick(int dtype, int d) {
  const int kind = kv_kind(dtype);
  if (is_bf16(dtype)) {
    if (d == 64) return kind == kKv16 ? K<__nv_bfloat16, 64, kKv16>::fn() : K<__nv_bfloat16, 64, kKvE2m1>::fn();
    return kind == kKv16 ? K<__nv_bfloat16, 128, kKv16>::fn() : K<__nv_bfloat16, 128, kKvE2m1>::fn();
  }
  if (d == 64)
    return kind == kKv16 ? K<__half, 64, kKv16>::fn()
           : kind == kKvE4m3 ? K<__half, 64, kKvE4m3>::fn() : K<__half, 64, kKvE2m1>::fn();
  return kind == kKv16 ? K<__half, 128, kKv16>::fn()
         : kind == kKvE4m3 ? K<__half, 128, kKvE4m3>::fn() : K<__half, 128, kKvE2m1>::fn();
}
template <typename T, int D, int KV>
struct AppendFn {
  static const void* fn() { return reinterpret_cast<const void*>(&fd_append_kernel<T, D, KV>); }
};
template <typename T, int D, int KV>
struct GatherFn {
  static const void* fn() { return reinterpret_cast<const void*>(&fd_gather_kernel<T, D, KV>); }
};

// Frequencies in units of 2^-64 turns per position (whole turns dropped), and their axes.
int set_rope(const fd_rope* rope, int d, bool four_bit_cache, AppendParams* p) {
  p->rot = 0;
  p->rope_scale = 1.f;
  if (rope == nullptr || rope->rot_dim == 0) return FD_OK;
  if (rope->rot_dim < 0 || rope->rot_dim > d || rope->rot_dim % 2 || rope->inv_freq == nullptr ||
      rope->num_axes < 1 || rope->num_axes > kMaxAxes || !std::isfinite(rope->scale) || rope->scale == 0.f)
    return FD_ERR_INVALID;
  if (rope->rot_dim % (four_bit_cache ? 32 : 16)) return FD_ERR_UNSUPPORTED;
  if (rope->num_axes > 1 && (p->positions == nullptr || p->pos_stride < p->T)) return FD_ERR_INVALID;
  for (int i = 0; i < rope->rot_dim / 2; ++i) {
    const double f = rope->inv_freq[i];
    if (!(std::fabs(f) <= kMaxFreq)) return FD_ERR_INVALID;  // NaN too
    // Turns per position in twice double precision (product and its rounding error), then
    // modulo 1 in 64 bits: the whole turns of the high part drop out exactly.
    const double high = f * 0.15915494309189535;                        // 1 / (2 pi), high part
    const double low = std::fma(f, 0.15915494309189535, -high) + f * -9.839338337591243e-18;
    const double part = std::fabs(high - std::trunc(high));
    const uint64_t units = (uint64_t)std::ldexp(part, 64);
    p->freq[i] = (high < 0 ? 0 - units : units) + (uint64_t)std::llrint(std::ldexp(low, 64));
    const int axis = rope->axis ? rope->axis[i] : 0;
    if (axis >= rope->num_axes) return FD_ERR_INVALID;
    p->axis[i] = (uint8_t)axis;
  }
  p->rot = rope->rot_dim;
  p->interleaved = rope->interleaved != 0;
  p->rope_scale = rope->scale;
  return FD_OK;
}

Span input_span(const void* p, const int64_t* stride, int64_t T, int H, int d) {
  return span(p, 2 * ((T - 1) * stride[0] + (H - 1) * stride[1] + d));
}
// Bytes of one cache.
int64_t cache_span(const fd_rows_s* r, int num_pages) {
  return r->page_size ? (int64_t)num_pages * r->cache_bytes : r->cache_bytes;
}
// Bytes of the page table that a call may read.
int64_t table_bytes(const fd_rows_s* r, int64_t bt_stride) { return 4 * ((r->B - 1) * bt_stride + r->max_pages); }
bool in_place(const void* out, const void* in, const int64_t* stride, int64_t T, int H, int d) {
  return out == in && (stride[1] == d || H == 1) && (stride[0] == (int64_t)H * d || T == 1);
}

}  // namespace
}  // namespace fd

extern "C" {

int fd_rows_plan(int B, int Hq, int Hkv, int d, const int32_t* seqlens, const int32_t* begin,
                 const int32_t* count, int page_size, int dtype, fd_rows_t* out_rows) {
  if (!out_rows) return FD_ERR_INVALID;
  *out_rows = nullptr;
  if (!seqlens || !begin || !count) return FD_ERR_INVALID;
  if (B < 1 || Hq < 1 || Hkv < 1 || d < 1 || page_size < 0 || Hq % Hkv != 0) return FD_ERR_INVALID;
  if (dtype != FD_F16 && dtype != FD_BF16 && dtype != FD_F16_E4M3KV && dtype != FD_F16_E2M1KV &&
      dtype != FD_BF16_E2M1KV)
    return FD_ERR_INVALID;
  if (page_size != 0 && (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))))
    return FD_ERR_UNSUPPORTED;
  if (B > FD_MAX_BATCH || (d != 64 && d != 128)) return FD_ERR_UNSUPPORTED;
  const int64_t limit = (int64_t)1 << 31;
  if ((int64_t)Hq + 2 * (int64_t)Hkv >= limit / FD_MAX_BATCH) return FD_ERR_UNSUPPORTED;
  const bool four = fd::kv_kind(dtype) == fd::kKvE2m1;
  int64_t T = 0, rows = 0;
  int max_pages = 0;
  for (int b = 0; b < B; ++b) {
    if (seqlens[b] < 0 || begin[b] < 0 || count[b] < 0 ||
        (int64_t)begin[b] + count[b] > (int64_t)seqlens[b])
      return FD_ERR_INVALID;
    T += count[b];
    const int64_t L = seqlens[b];
    rows += four ? (L + fd::kBlockTokens - 1) / fd::kBlockTokens * fd::kBlockTokens : L;
    if (page_size) max_pages = (int)std::max<int64_t>(max_pages, (L + page_size - 1) / page_size);
  }
  if (rows >= limit) return FD_ERR_UNSUPPORTED;

  fd_rows_s* r = new (std::nothrow) fd_rows_s();
  if (!r) return FD_ERR_NOMEM;
  r->B = B; r->Hq = Hq; r->Hkv = Hkv; r->d = d; r->dtype = dtype; r->page_size = page_size;
  r->max_pages = max_pages;
  r->T = T;
  r->cache_bytes = (page_size ? page_size : rows) * Hkv * fd::row_bytes(r);
  int32_t cu = 0, base = 0;
  for (int b = 0; b < B; ++b) {
    r->cu[b] = cu;
    r->begin[b] = begin[b];
    r->base[b] = base;
    cu += count[b];
    base += four ? (int32_t)(((int64_t)seqlens[b] + fd::kBlockTokens - 1) / fd::kBlockTokens * fd::kBlockTokens)
                 : seqlens[b];
  }
  r->cu[B] = cu;
  *out_rows = r;
  return FD_OK;
}

int fd_rows_destroy(fd_rows_t rows) {
  delete rows;
  return FD_OK;
}

int fd_rows_get_info(fd_rows_t rows, fd_rows_info* info) {
  if (!rows || !info) return FD_ERR_INVALID;
  info->tokens = rows->T;
  info->cache_bytes = rows->cache_bytes;
  return FD_OK;
}

int fd_append(fd_rows_t rows, const fd_append_args* a, cudaStream_t stream) {
  if (!rows || !a) return FD_ERR_INVALID;
  const fd_rows_s* r = rows;
  const int d = r->d, kind = fd::kv_kind(r->dtype);
  if ((a->q != nullptr) != (a->q_out != nullptr) || (a->v != nullptr) != (a->v_cache != nullptr) ||
      (a->k_cache != nullptr) != (a->v_cache != nullptr) ||
      (a->k != nullptr) != (a->k_out != nullptr || a->k_cache != nullptr) || (!a->q && !a->k))
    return FD_ERR_INVALID;
  const int64_t* strides[3] = {a->q_stride, a->k_stride, a->v_stride};
  const void* ins[3] = {a->q, a->k, a->v};
  for (int i = 0; i < 3; ++i)
    if (ins[i] && (strides[i][0] < 0 || strides[i][1] < 0)) return FD_ERR_INVALID;
  if (a->k_cache) {
    if (!std::isfinite(a->k_mul) || !std::isfinite(a->v_mul) || a->k_mul <= 0.f || a->v_mul <= 0.f)
      return FD_ERR_INVALID;
    if (kind == fd::kKv16 && (a->k_mul != 1.f || a->v_mul != 1.f)) return FD_ERR_INVALID;
  }
  if ((a->q_norm || a->k_norm) &&
      (!std::isfinite(a->eps) || a->eps < 0.f || !std::isfinite(a->weight_offset)))
    return FD_ERR_INVALID;
  for (const void* p : {a->q, a->k, a->v, a->q_weight, a->k_weight, (const void*)a->q_out,
                        (const void*)a->k_out, (const void*)a->k_cache, (const void*)a->v_cache})
    if (!fd::aligned(p, 16)) return FD_ERR_ALIGN;
  if (!fd::aligned(a->positions, 4)) return FD_ERR_ALIGN;
  for (int i = 0; i < 3; ++i)
    if (ins[i] && (strides[i][0] % 8 || strides[i][1] % 8)) return FD_ERR_ALIGN;

  fd::AppendParams p;
  p.T = (int32_t)r->T;
  p.positions = a->positions;
  p.pos_stride = a->pos_stride;
  p.interleaved = 0;
  int rc = fd::set_rope(a->rope, d, kind == fd::kKvE2m1 && a->k_cache, &p);
  if (rc != FD_OK) return rc;
  if (a->k_cache) {
    rc = fd::make_map(r, a->num_pages, a->block_table, a->bt_stride, a->status, &p.m);
    if (rc != FD_OK) return rc;
  } else {
    // Nothing is stored in a cache: the map only tells rows (default positions) from tokens.
    fd_rows_s flat = *r;
    flat.page_size = 0;
    rc = fd::make_map(&flat, 0, nullptr, 0, nullptr, &p.m);
    if (rc != FD_OK) return rc;
  }
  const int64_t T = r->T;
  if (T == 0) return FD_OK;
  const int heads[3] = {r->Hq, r->Hkv, r->Hkv};
  const int64_t cache = a->k_cache ? fd::cache_span(r, a->num_pages) : 0;
  const int64_t axes = p.rot > 0 && a->positions ? a->rope->num_axes : 0;
  const fd::Span outs[5] = {fd::span(a->q_out, 2 * T * r->Hq * d), fd::span(a->k_out, 2 * T * r->Hkv * d),
                            fd::span(a->k_cache, cache), fd::span(a->v_cache, cache),
                            fd::span(a->k_cache ? a->status : nullptr, 4)};
  // q, k and v first.
  const fd::Span reads[7] = {fd::input_span(a->q, a->q_stride, T, r->Hq, d), fd::input_span(a->k, a->k_stride, T, r->Hkv, d),
                             fd::input_span(a->v, a->v_stride, T, r->Hkv, d),
                             fd::span(a->q_norm ? a->q_weight : nullptr, 2 * d),
                             fd::span(a->k_norm ? a->k_weight : nullptr, 2 * d),
                             fd::span(axes ? a->positions : nullptr, 4 * ((axes - 1) * a->pos_stride + T)),
                             fd::span(p.m.block_table, fd::table_bytes(r, a->bt_stride))};
  for (int o = 0; o < 5; ++o) {
    for (int i = 0; i < 7; ++i) {
      // q_out may be q and k_out k, element for element.
      if (o == i && o < 2 && fd::in_place(o ? a->k_out : a->q_out, ins[i], strides[i], T, heads[i], d)) continue;
      if (fd::overlap(outs[o], reads[i])) return FD_ERR_INVALID;
    }
    for (int k = 0; k < o; ++k)
      if (fd::overlap(outs[o], outs[k])) return FD_ERR_INVALID;
  }
  p.q = a->q; p.k = a->k; p.v = a->v;
  p.q_weight = a->q_weight; p.k_weight = a->k_weight;
  std::memcpy(p.q_stride, a->q_stride, sizeof(p.q_stride));
  std::memcpy(p.k_stride, a->k_stride, sizeof(p.k_stride));
  std::memcpy(p.v_stride, a->v_stride, sizeof(p.v_stride));
  p.q_out = a->q_out; p.k_out = a->k_out; p.k_cache = a->k_cache; p.v_cache = a->v_cache;
  p.eps = a->eps;
  p.weight_offset = a->weight_offset;
  p.k_mul = a->k_mul; p.v_mul = a->v_mul;
  p.q_norm = a->q_norm != 0; p.k_norm = a->k_norm != 0;
  p.Hq = r->Hq;
  // Head rows per warp: one round (4 rows at d = 128) while tokens are few, so that a decode step
  // fills the device; more as they grow, so that the angles of a token are computed less often.
  const int rows_all = (a->q ? r->Hq : 0) + (a->k ? r->Hkv : 0) + (a->v ? r->Hkv : 0);
  const int round = 512 / d;
  int64_t per = (T * rows_all + fd::kAppendWarps - 1) / fd::kAppendWarps;
  per = (per + round - 1) / round * round;
  if (per > rows_all) per = rows_all;
  p.rows_per_warp = (int32_t)per;
  p.splits = (int32_t)((rows_all + per - 1) / per);
  return fd::launch_rows(fd::pick<fd::AppendFn>(r->dtype, d), T * p.splits, &p, stream);
}

int fd_gather(fd_rows_t rows, const void* k_cache, const void* v_cache, int num_pages,
              const int32_t* block_table, int bt_stride, void* k_out, void* v_out,
              uint32_t* status, cudaStream_t stream) {
  if (!rows || !k_cache || !v_cache || !k_out || !v_out) return FD_ERR_INVALID;
  for (const void* p : {k_cache, v_cache, (const void*)k_out, (const void*)v_out})
    if (!fd::aligned(p, 16)) return FD_ERR_ALIGN;
  fd::GatherParams p;
  int rc = fd::make_map(rows, num_pages, block_table, bt_stride, status, &p.m);
  if (rc != FD_OK) return rc;
  if (rows->T == 0) return FD_OK;
  const int64_t cache = fd::cache_span(rows, num_pages), bytes = 2 * rows->T * rows->Hkv * rows->d;
  const fd::Span outs[3] = {fd::span(k_out, bytes), fd::span(v_out, bytes), fd::span(status, 4)};
  const fd::Span reads[3] = {fd::span(k_cache, cache), fd::span(v_cache, cache),
                             fd::span(block_table, fd::table_bytes(rows, bt_stride))};
  for (int o = 0; o < 3; ++o) {
    for (const fd::Span& in : reads)
      if (fd::overlap(outs[o], in)) return FD_ERR_INVALID;
    for (int k = 0; k < o; ++k)
      if (fd::overlap(outs[o], outs[k])) return FD_ERR_INVALID;
  }
  p.k_cache = k_cache; p.v_cache = v_cache;
  p.k_out = k_out; p.v_out = v_out;
  p.T = (int32_t)rows->T;
  const int64_t tok = fd::gather_tokens(rows->d), tiles = (rows->T + tok - 1) / tok;
  return fd::launch_rows(fd::pick<fd::GatherFn>(rows->dtype, rows->d), tiles * 2 * rows->Hkv, &p, stream);
}

}  // extern "C"
