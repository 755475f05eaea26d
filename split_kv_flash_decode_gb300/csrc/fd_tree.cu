// A step of speculative decoding: the plan, the verdict on drafted tokens (fd_tree_verify) and the
// rows that stand (fd_tree_keep).  The attention is in fd_tree_attn.cuh.  See fd.h for the contract.
#include "fd_tree.h"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "fd_kernel.cuh"
#include "fd_plan_internal.h"

namespace fd {
namespace {

// ------------------------------------------------------------------ verify

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCluster = 8;  // CTAs of a sequence: each reads a slice of its row

struct VerifyParams {
  const float *target, *draft;
  int64_t target_stride, draft_stride;
  const int32_t *tokens, *parents;
  const float* uniform;
  int32_t *path, *emitted, *count;
  int32_t vocab, max_drafts;
  int32_t cu[FD_MAX_BATCH + 1];
};

// A probability as it counts: NaN as 0.
__device__ __forceinline__ float weight(float x) { return __saturatef(x); }
// A value in [0, 16) in units of 2^-57 (below 2^-34 its last bits are cut): the significand, shifted by what the
// exponent says.  (The conversion instruction to 64 bits runs at the rate of fp64.)
__device__ __forceinline__ uint64_t fixed_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return (uint64_t)((b << 5 & 0x0fffffe0u) | 0x10000000u) << 32 >> min(130 - (b >> 23), 63u);
}
__device__ __forceinline__ uint64_t fixed(float x) { return fixed_of(weight(x)); }
// Sums of rows that are no probabilities (logits, say) stop here, so that none of them wraps around: 64 warps' sums, and
// what the search adds to one of them, stay within 64 bits.
constexpr uint64_t kMost = (1ull << 60) - 1;
__device__ __forceinline__ uint64_t plus_most(uint64_t a, uint64_t b) { return min(a + b, kMost); }
// A thread's sum of weights: two running sums (of the even and the odd ones) with what their additions and differences
// rounded away beside them, so that some dozens of weights are off by 2^-46 of their sum.  All on the fp32 pipe, two
// values an instruction; in 64-bit integers the sums took longer than the rows' bytes (64 rows of 131072 of both: 25 us).
struct Sum {
  uint64_t high = 0, low = 0;
  static __device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
  }
  static __device__ __forceinline__ float2 unpair(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
  }
  static __device__ __forceinline__ uint64_t plus(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
  }
  static __device__ __forceinline__ uint64_t minus(uint64_t a, uint64_t b) {  // a - b, rounded once
    uint64_t r;
    asm("{\n\t.reg .b64 m;\n\tmov.b64 m, 0xbf800000bf800000;\n\tfma.rn.f32x2 %0, %2, m, %1;\n\t}" : "=l"(r) : "l"(a), "l"(b));
    return r;
  }
  // The sum and its rounding error (Knuth).
  __device__ __forceinline__ void accumulate(uint64_t w, uint64_t e) {
    const uint64_t s = plus(high, w), z = minus(s, high);
    low = plus(low, plus(plus(minus(high, minus(s, z)), minus(w, z)), e));
    high = s;
  }
  __device__ __forceinline__ void add(float a, float b) { accumulate(pair(weight(a), weight(b)), 0); }
  // max(a - qa, 0) and max(b - qb, 0): the difference and its rounding error, or neither.
  __device__ __forceinline__ void add_left(float a, float qa, float b, float qb) {
    const uint64_t x = pair(weight(a), weight(b)), y = pair(weight(qa), weight(qb));
    const uint64_t s = minus(x, y), v = minus(s, x);
    const float2 d = unpair(s), e = unpair(minus(minus(x, minus(s, v)), plus(y, v)));
    accumulate(pair(fmaxf(d.x, 0.f), fmaxf(d.y, 0.f)), pair(d.x > 0.f ? e.x : 0.f, d.y > 0.f ? e.y : 0.f));
  }
  // In units of 2^-57.
  __device__ __forceinline__ uint64_t fixed_sum() const {
    const float2 h = unpair(high), l = unpair(low);
    const float rest = fminf(fmaxf(l.x + l.y, -8.f), 8.f);
    const uint64_t sum = fixed_of(fminf(h.x, 8.f)) + fixed_of(fminf(h.y, 8.f)), r = fixed_of(fabsf(rest));
    return min(rest >= 0.f ? sum + r : sum > r ? sum - r : 0, kMost);
  }
};
__device__ __forceinline__ uint64_t less(uint64_t a, uint64_t b) { return a > b ? a - b : 0; }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Store into the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void store_cluster_u64(uint32_t addr, uint32_t rank, uint64_t v) {
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
               "st.shared::cluster.u64 [a], %2;\n\t}" ::"r"(addr), "r"(rank), "l"(v) : "memory");
}

// One cluster per sequence.  The walk is the same in every CTA: a lane holds two nodes, with the target's
// probability of their tokens (all gathered at once: the walk's chain is one load long), and a ballot finds
// the children of a node.  Then each CTA sums a slice of the last node's row, the cluster adds the slices up,
// and the CTA in whose slice the draw falls looks for it there.
//
// Bound by latency but for many sequences: a launch, the walk's gather, one batch of loads per thread, a cluster
// barrier, the search.  One tree over 32768 tokens 5.4 us, 17 over 50021 (whose
// rows begin at odd places) 9.2; 64 chains of 131072 tokens with both rows
// 19.0 us, 3.5 TB/s.  There each cluster reads one row after its walk, in one wave; 512 threads a CTA, loads that pass
// the L1 and 64-bit integer sums (25 us) were not faster.
__global__ void __launch_bounds__(kVerifyThreads) __cluster_dims__(kVerifyCluster, 1, 1)
    fd_verify_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ int32_t tokens[FD_MAX_DRAFTS];
  __shared__ uint64_t warp_sum[2][kVerifyWarps];
  __shared__ uint64_t slice_sum[2][kVerifyCluster];
  __shared__ uint64_t stands_s, tried_s;
  __shared__ int last_s;
  dev::pdl_launch_dependents();
  dev::pdl_wait();
  const int b = blockIdx.x / kVerifyCluster, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int first = p.cu[b], n = p.cu[b + 1] - first, V = p.vocab;
  if (n == 0) {
    if (rank == 0) {
      for (int i = tid; i < p.max_drafts; i += kVerifyThreads)
        p.path[(int64_t)b * p.max_drafts + i] = p.emitted[(int64_t)b * p.max_drafts + i] = -1;
      if (tid == 0) p.count[b] = 0;
    }
    return;
  }
  cluster_arrive();  // this CTA runs, so that others may write its shared memory
  if (warp == 0) {
    int up[2], tok[2];
    float u[2], pt[2], qt[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = lane + 32 * k;
      up[k] = tok[k] = -1;
      u[k] = pt[k] = qt[k] = 0.f;
      if (i < n) {
        tok[k] = p.tokens[first + i];
        tokens[i] = tok[k];
        u[k] = p.uniform[first + i];
        const int parent = p.parents != nullptr ? p.parents[first + i] : i - 1;
        if (i > 0 && parent >= 0 && parent < i) {
          up[k] = parent;
          if ((uint32_t)tok[k] < (uint32_t)V) {
            pt[k] = weight(p.target[(first + parent) * p.target_stride + tok[k]]);
            if (p.draft != nullptr) qt[k] = weight(p.draft[(first + i) * p.draft_stride + tok[k]]);
          }
        }
      }
    }
    auto bits = [&](bool a, bool b) {
      const uint32_t lo = __ballot_sync(0xffffffffu, a), hi = __ballot_sync(0xffffffffu, b);
      return (uint64_t)hi << 32 | lo;
    };
    uint64_t stands = 1, tried = 0;
    int node = 0;
    for (;;) {  // at most n rounds: a child lies above its parent
      uint64_t below = bits(up[0] == node, up[1] == node);
      double mass = 1.0;
      int went = -1;
      tried = 0;
      while (below != 0) {
        const int i = __ffsll((long long)below) - 1, src = i & 31;
        below &= below - 1;
        const float pi = __shfl_sync(0xffffffffu, i < 32 ? pt[0] : pt[1], src);
        const float ui = __shfl_sync(0xffffffffu, i < 32 ? u[0] : u[1], src);
        // A probability of 0 is looked at by itself: beside a random number outside [0, 1) a product can be below it.
        if (p.draft != nullptr) {
          const float qi = __shfl_sync(0xffffffffu, i < 32 ? qt[0] : qt[1], src);
          if (pi > 0.f && (double)ui * (double)qi < (double)pi) went = i;
        } else {
          const int ti = __shfl_sync(0xffffffffu, i < 32 ? tok[0] : tok[1], src);
          const uint64_t same = bits(tok[0] == ti, tok[1] == ti);
          const float left = (same & tried) ? 0.f : pi;
          if (left > 0.f && (double)ui * mass < (double)left) went = i;
          else mass -= (double)left;
        }
        if (went >= 0) break;
        tried |= 1ull << i;
      }
      if (went < 0) break;
      node = went;
      stands |= 1ull << node;
    }
    if (lane == 0) {
      stands_s = stands;
      tried_s = tried;
    }
    if (rank == 0) {
      const int count = __popcll(stands);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = lane + 32 * k;
        if ((stands >> i) & 1) {
          const int at = __popcll(stands & ((1ull << i) - 1));
          p.path[(int64_t)b * p.max_drafts + at] = i;
          if (at > 0) p.emitted[(int64_t)b * p.max_drafts + at - 1] = tok[k];
        }
        if (i >= count && i < p.max_drafts)
          p.path[(int64_t)b * p.max_drafts + i] = p.emitted[(int64_t)b * p.max_drafts + i] = -1;
      }
      if (lane == 0) p.count[b] = count;
    }
  }
  __syncthreads();
  const uint64_t stands = stands_s, tried = tried_s;
  const int node = 63 - __clzll((long long)stands);
  const float u0 = p.uniform[first];
  const float* target = p.target + (first + node) * p.target_stride;
  // The slice of this CTA, and this warp's part of it.
  constexpr int kParts = kVerifyCluster * kVerifyWarps, kStep = 128;
  const int per_warp = ((V + kParts - 1) / kParts + kStep - 1) / kStep * kStep;
  const int c0 = min((int)rank * kVerifyWarps * per_warp, V), c1 = min(c0 + kVerifyWarps * per_warp, V);
  const int w0 = min(c0 + warp * per_warp, c1), w1 = min(w0 + per_warp, c1);

  for (int attempt = 0;; ++attempt) {
    // The second attempt draws from the target itself: nothing was left.
    const bool rest = attempt == 0 && tried != 0;
    const float* draft = rest && p.draft != nullptr ? p.draft + (first + __ffsll((long long)tried) - 1) * p.draft_stride : nullptr;
    const uint64_t gone = rest && p.draft == nullptr ? tried : 0;
    Sum part;
    int at0 = w0 + lane;
    // 16 bytes at a time where both rows allow it.  (Plain loads: the read-only path is for memory that nobody writes while
    // the kernel runs, and this one may begin while a kernel before it still writes the rows.)
    if (((reinterpret_cast<uintptr_t>(target) | reinterpret_cast<uintptr_t>(draft)) & 15) == 0) {
      const int whole = w1 & ~3;
      if (draft != nullptr) {
#pragma unroll 4
        for (int i = w0 + 4 * lane; i < whole; i += kStep) {
          const float4 a = *reinterpret_cast<const float4*>(target + i), b = *reinterpret_cast<const float4*>(draft + i);
          part.add_left(a.x, b.x, a.y, b.y);
          part.add_left(a.z, b.z, a.w, b.w);
        }
      } else {
#pragma unroll 4
        for (int i = w0 + 4 * lane; i < whole; i += kStep) {
          const float4 a = *reinterpret_cast<const float4*>(target + i);
          part.add(a.x, a.y);
          part.add(a.z, a.w);
        }
      }
      at0 = max(w0, whole) + lane;
    }
#pragma unroll 4
    for (int i = at0; i < w1; i += 64) {
      const int j = min(i + 32, w1 - 1);                 // past the end: weighs nothing
      const float a = target[i], b = i + 32 < w1 ? target[j] : 0.f;
      if (draft != nullptr) part.add_left(a, draft[i], b, i + 32 < w1 ? draft[j] : 0.f);
      else part.add(a, b);
    }
    uint64_t sum = part.fixed_sum(), away = 0;
    // Tokens that were tried weigh nothing; one that was tried twice goes once.
    for (uint64_t m = gone; m != 0; m &= m - 1) {
      const int i = __ffsll((long long)m) - 1, t = tokens[i];
      bool again = false;
      for (uint64_t e = gone & ((1ull << i) - 1); e != 0; e &= e - 1) again |= tokens[__ffsll((long long)e) - 1] == t;
      if (t >= w0 && t < w1 && !again) away += fixed(target[t]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum = plus_most(sum, __shfl_xor_sync(0xffffffffu, sum, off));
    // What the tried tokens leave must be more than the roundings of both sums (3 units a lane, one a token, 2^-46 of
    // the whole): else nothing is left, and nothing could be found.
    if (lane == 0) warp_sum[attempt][warp] = gone == 0 ? sum : sum > away + (sum >> 44) + 256 ? sum - away : 0;
    __syncthreads();
    if (attempt == 0) cluster_wait();
    if (tid < kVerifyCluster) {
      uint64_t all = 0;
      for (int w = 0; w < kVerifyWarps; ++w) all = plus_most(all, warp_sum[attempt][w]);
      store_cluster_u64(dev::smem_addr(&slice_sum[attempt][rank]), tid, all);
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    uint64_t total = 0, before = 0;
    for (int r = 0; r < kVerifyCluster; ++r) {
      before += r < (int)rank ? slice_sum[attempt][r] : 0;
      total += slice_sum[attempt][r];
    }
    if (total == 0) {
      if (rest) continue;
      if (rank == 0 && tid == 0) p.emitted[(int64_t)b * p.max_drafts + __popcll(stands) - 1] = -1;
      return;
    }
    // The first token with a sum up to it over uniform x total.
    const uint64_t r64 = u0 >= 1.f ? ~0ull : u0 > 0.f ? __double2ull_rz((double)u0 * 0x1p64) : 0;
    const uint64_t at = __umul64hi(total, r64);
    if (at < before || at >= before + slice_sum[attempt][rank]) return;
    int w = 0;
    while (at >= before + warp_sum[attempt][w]) before += warp_sum[attempt][w++];
    const int s0 = min(c0 + w * per_warp, c1), s1 = min(s0 + per_warp, c1);
    int heavy = -1;  // this thread's last token with a weight
    if (tid == 0) last_s = -1;
    // All threads look through that warp's part: eight tokens each.
    for (int at0 = s0; at0 < s1; at0 += 8 * kVerifyThreads) {
      uint64_t x[8], mine = 0;
      uint32_t weighs = 0;
      const int i0 = at0 + 8 * tid;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + k;
        const float a = i < s1 ? weight(target[i]) : 0.f, b = draft != nullptr && i < s1 ? weight(draft[i]) : 0.f;
        x[k] = less(fixed_of(a), fixed_of(b));
        if (a > b) weighs |= 1u << k;
      }
      for (uint64_t m = gone; m != 0; m &= m - 1) {
        const int t = tokens[__ffsll((long long)m) - 1] - i0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (t == k) {
            x[k] = 0;
            weighs &= ~(1u << k);
          }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) mine += x[k];
      if (weighs != 0) heavy = i0 + 31 - __clz(weighs);
      uint64_t upto = min(mine, kMost);
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint64_t o = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto = plus_most(upto, o);
      }
      __syncthreads();  // the sums of the last round are read
      if (lane == 31) warp_sum[attempt ^ 1][warp] = upto;
      __syncthreads();
      uint64_t sum0 = before;
      for (int k = 0; k < kVerifyWarps; ++k) {
        if (k < warp) sum0 += warp_sum[attempt ^ 1][k];
        before += warp_sum[attempt ^ 1][k];
      }
      const uint64_t end = sum0 + upto, left = __shfl_up_sync(0xffffffffu, upto, 1);
      sum0 += lane > 0 ? left : 0;
      if (at >= sum0 && at < end) {
        int k = 0;
#pragma unroll
        for (int j = 0; j < 7; ++j) {
          if (k == j && at >= sum0 + x[j]) {
            sum0 += x[j];
            k = j + 1;
          }
        }
        p.emitted[(int64_t)b * p.max_drafts + __popcll(stands) - 1] = i0 + k;
      }
      if (at < before) return;  // the same in every thread
    }
    // The weights one by one came to less than their sum (by 2^-46 of it, or units that each of them lacks): the last.
    if (heavy >= 0) atomicMax(&last_s, heavy);
    __syncthreads();
    if (tid == 0) p.emitted[(int64_t)b * p.max_drafts + __popcll(stands) - 1] = last_s;
    return;
  }
}

// ------------------------------------------------------------------ keep

constexpr int kKeepThreads = 128;

struct KeepParams {
  uint8_t *k_cache, *v_cache;
  const int32_t *block_table, *path, *count;
  uint32_t* status;
  int32_t Hkv, d, page_shift, num_pages, bt_stride, path_stride, pieces;
  int32_t cu[FD_MAX_BATCH + 1];
  int32_t first[FD_MAX_BATCH];  // row of node 0 in its sequence
  int32_t base[FD_MAX_BATCH];
};

// Moves one piece of n rows; where(row) is the piece's place in the cache.  Sources lie behind their
// destinations, so a batch of loads ahead of its stores never reads what was written.
template <typename W, typename F>
__device__ __forceinline__ void move_rows(uint8_t* cache, const int64_t* from, const int64_t* to, int n, F where) {
  constexpr int kBatch = 8;
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    W x[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i0 + k < n && from[i0 + k] >= 0) x[k] = *reinterpret_cast<const W*>(cache + where(from[i0 + k]));
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i0 + k < n && from[i0 + k] >= 0) *reinterpret_cast<W*>(cache + where(to[i0 + k])) = x[k];
  }
}

// One thread: one piece of K (even blocks of a sequence) or V of a row, through all rows of its sequence
// that move: nothing is shared between threads, so the move needs no order among them.  Pieces are 16
// bytes; of a 4-bit block, whose rows lie in parts, 4 bytes, and single bytes for V's scales.  Bound by the
// launch and two loads in series (the page's index, then the rows): 2.4 us for one sequence, 4.8 for 64 of E4M3.
template <int KV>
__global__ void __launch_bounds__(kKeepThreads) fd_keep_kernel(const __grid_constant__ KeepParams p) {
  __shared__ int64_t from[FD_MAX_DRAFTS], to[FD_MAX_DRAFTS];
  __shared__ int bad[2];
  dev::pdl_launch_dependents();
  dev::pdl_wait();
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int n = p.cu[b + 1] - p.cu[b];
  const int count = min(max(p.count[b], 0), n);
  if (count == 0) return;
  auto row_of = [&](int r) {
    r += p.first[b];
    if (p.block_table == nullptr) return (int64_t)p.base[b] + r;
    const int pg = p.block_table[(int64_t)b * p.bt_stride + (r >> p.page_shift)];
    if ((uint32_t)pg >= (uint32_t)p.num_pages) {
      if (p.status != nullptr) atomicOr(p.status, FD_TREE_BAD_PAGE);
      return (int64_t)-1;
    }
    return ((int64_t)pg << p.page_shift) + (r & ((1 << p.page_shift) - 1));
  };
  if (tid < FD_MAX_DRAFTS) {
    const int32_t* path = p.path + (int64_t)b * p.path_stride;
    const int node = tid < count ? path[tid] : -1;
    const bool ascends = node >= 0 && node < n && (tid == 0 || node > path[tid - 1]);
    const uint32_t wrong = __ballot_sync(0xffffffffu, tid < count && !ascends);
    if (lane == 0) bad[tid >> 5] = wrong != 0 ? tid + __ffs(wrong) - 1 : FD_MAX_DRAFTS;
    int64_t src = -1, dst = -1;
    if (tid < count && ascends && node != tid) {
      src = row_of(node);
      dst = row_of(tid);
    }
    from[tid] = dst < 0 ? -1 : src;
    to[tid] = dst;
  }
  __syncthreads();
  const int good = min(bad[0], bad[1]), rows = min(count, good);
  if (good < count && p.status != nullptr && tid == 0) atomicOr(p.status, FD_TREE_BAD_PATH);
  const bool is_v = blockIdx.x & 1;
  const int piece = (blockIdx.x >> 1) * kKeepThreads + tid;
  if (piece >= p.pieces) return;
  uint8_t* cache = is_v ? p.v_cache : p.k_cache;
  const int d = p.d;
  if constexpr (KV != kKvE2m1) {
    const int64_t row_bytes = (int64_t)p.Hkv * d * (KV == kKv16 ? 2 : 1);
    move_rows<uint4>(cache, from, to, rows, [&](int64_t row) { return row * row_bytes + 16 * piece; });
  } else {
    // Pieces of a KV head: d / 8 of codes, then its scales: d / 16 bytes, of K together, of V 16 apart.
    const int per_head = d / 8 + d / 16, h = piece / per_head, i = piece - h * per_head;
    const int64_t block_bytes = (int64_t)p.Hkv * 9 * d;
    cache += (int64_t)h * 9 * d;
    if (i < d / 8) {
      // V: piece i lies in group i / (d / 64) of d / 8 elements.
      const int g = i / (d / 64), swap = ((d == 128 ? g : g >> 1) & 1) << 2, part = 4 * (i - g * (d / 64));
      move_rows<uint32_t>(cache, from, to, rows, [&](int64_t row) {
        const int r = (int)(row & (kBlockTokens - 1));
        return (row >> kBlockShift) * block_bytes +
               (is_v ? g * d + ((r >> 1) ^ swap) * (d / 8) + (r & 1) * (d / 16) + part : r * (d / 2) + 4 * i);
      });
    } else {
      const int j = i - d / 8;
      move_rows<uint8_t>(cache, from, to, rows, [&](int64_t row) {
        const int r = (int)(row & (kBlockTokens - 1));
        return (row >> kBlockShift) * block_bytes + 8 * d + (is_v ? 16 * j + r : r * (d / 16) + j);
      });
    }
  }
}

// ------------------------------------------------------------------ host

int launch(const void* fn, dim3 grid, int threads, const void* params, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void* args[] = {const_cast<void*>(params)};
  if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) {
    cudaGetLastError();
    return FD_ERR_CUDA;
  }
  return FD_OK;
}

// Page-table arguments of a call; sets the page's bits.
int check_pages(const fd_tree_s* t, int num_pages, const int32_t* block_table, int bt_stride, int32_t* shift) {
  *shift = 0;
  if (!t->page_size) return block_table != nullptr ? FD_ERR_INVALID : FD_OK;
  if (num_pages < 1 || block_table == nullptr || bt_stride < t->max_pages) return FD_ERR_INVALID;
  if ((int64_t)num_pages * t->page_size >= (int64_t)1 << 31) return FD_ERR_UNSUPPORTED;
  while ((1 << *shift) < t->page_size) ++*shift;
  return FD_OK;
}
int64_t cache_rows(const fd_tree_s* t, int num_pages) {
  if (t->page_size) return (int64_t)num_pages * t->page_size;
  return kv_kind(t->dtype) == kKvE2m1 ? t->n_blocks * kBlockTokens : t->n_tokens;
}
Span cache_span(const fd_tree_s* t, const void* p, int num_pages) {
  return span(p, cache_rows(t, num_pages) * t->Hkv * cache_row_bytes(t->dtype, t->d));
}
Span table_span(const fd_tree_s* t, const int32_t* table, int64_t bt_stride) {
  return span(table, 4 * ((t->B - 1) * bt_stride + t->max_pages));
}
// The 3-D view of a cache that the attention's loads take: (d, Hkv, rows); 16 bits in boxes of 64 columns with
// the 128-byte swizzle, as the tensor cores read them, E4M3 in whole rows, 4 bits in whole blocks.
int encode_cache(CUtensorMap* map, const fd_tree_s* t, const void* cache, int num_pages) {
  const int kind = kv_kind(t->dtype), d = t->d, unit = kind == kKvE2m1 ? kBlockTokens : 1;
  const cuuint64_t row = (cuuint64_t)cache_row_bytes(t->dtype, d) * unit;
  const cuuint64_t dims[3] = {(cuuint64_t)(kind == kKvE2m1 ? 9 * d / 8 : d), (cuuint64_t)t->Hkv,
                              (cuuint64_t)(cache_rows(t, num_pages) / unit)};
  const cuuint64_t strides[2] = {row, row * t->Hkv};
  const cuuint32_t box[3] = {(cuuint32_t)(kind == kKv16   ? 64
                                          : kind == kKvE4m3 ? d
                                                            : ring_row_bytes(kPathMmaKv4, d) * kBlockTokens / 8),
                             1u, (cuuint32_t)(t->params.box_rows / unit)};
  return encode_map(map,
                    kind == kKvE4m3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                    : kind == kKvE2m1 ? CU_TENSOR_MAP_DATA_TYPE_UINT64
                    : is_bf16(t->dtype) ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                    cache, dims, strides, box, kind == kKv16 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                    // A head's row: its neighbours are other heads', which other CTAs read at other times.
                    row >= 256 && kind != kKvE2m1 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                    : row >= 128                  ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                  : CU_TENSOR_MAP_L2_PROMOTION_L2_64B);
}
// Whether an output overlaps an input or another output.
template <size_t N, size_t M>
bool any_overlap(const Span (&outs)[N], const Span (&ins)[M]) {
  for (size_t o = 0; o < N; ++o) {
    for (const Span& i : ins)
      if (overlap(outs[o], i)) return true;
    for (size_t k = 0; k < o; ++k)
      if (overlap(outs[o], outs[k])) return true;
  }
  return false;
}

}  // namespace
}  // namespace fd

extern "C" {

int fd_tree_plan(int B, int Hq, int Hkv, int d, const int32_t* seqlens, const int32_t* drafts, int page_size,
                 int dtype, int num_sms, fd_tree_t* out_tree) {
  if (!out_tree) return FD_ERR_INVALID;
  *out_tree = nullptr;
  if (!seqlens || !drafts) return FD_ERR_INVALID;
  if (B < 1 || Hq < 1 || Hkv < 1 || d < 1 || page_size < 0 || num_sms < 0 || Hq % Hkv != 0) return FD_ERR_INVALID;
  if (dtype != FD_F16 && dtype != FD_BF16 && dtype != FD_F16_E4M3KV && dtype != FD_F16_E2M1KV &&
      dtype != FD_BF16_E2M1KV)
    return FD_ERR_INVALID;
  if (page_size != 0 && (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))))
    return FD_ERR_UNSUPPORTED;
  if (B > FD_MAX_BATCH || (d != 64 && d != 128)) return FD_ERR_UNSUPPORTED;
  const int64_t limit = (int64_t)1 << 31;
  // Query rows of a sequence (64 x Hq / Hkv) and pieces of a row stay far within 32 bits.
  if (Hq > 4096) return FD_ERR_UNSUPPORTED;
  const bool four = fd::kv_kind(dtype) == fd::kKvE2m1;
  int64_t T = 0, tokens = 0, blocks = 0, read = 0;
  int max_pages = 0, max_drafts = 0;
  for (int b = 0; b < B; ++b) {
    if (seqlens[b] < 0 || drafts[b] < 0 || drafts[b] > seqlens[b]) return FD_ERR_INVALID;
    if (drafts[b] > FD_MAX_DRAFTS) return FD_ERR_UNSUPPORTED;
    T += drafts[b];
    tokens += seqlens[b];
    blocks += ((int64_t)seqlens[b] + fd::kBlockTokens - 1) / fd::kBlockTokens;
    if (drafts[b]) read += seqlens[b];
    max_drafts = std::max(max_drafts, (int)drafts[b]);
    if (page_size) max_pages = std::max(max_pages, (int)(((int64_t)seqlens[b] + page_size - 1) / page_size));
  }
  if ((four ? blocks * fd::kBlockTokens : tokens) >= limit) return FD_ERR_UNSUPPORTED;
  if (num_sms == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return FD_ERR_CUDA;
    }
  }
  // Units of work: the tiles of every item, and what an item costs beyond them.
  const int G = Hq / Hkv;
  int64_t tiles = 0, all_items = 0;
  int rows = 0, longest = 0;
  for (int b = 0; b < B; ++b) {
    if (!drafts[b]) continue;
    const int64_t items = (int64_t)Hkv * fd::tree_groups(drafts[b] * G);
    tiles += items * fd::tree_tiles(seqlens[b]);
    all_items += items;
    longest = std::max(longest, fd::tree_tiles(seqlens[b]));
    rows = std::max(rows, drafts[b] * G);
  }
  if (tiles + all_items * fd::kTreeMaxItemUnits >= limit) return FD_ERR_UNSUPPORTED;
  fd_tree_s* t = new (std::nothrow) fd_tree_s();
  if (!t) return FD_ERR_NOMEM;
  t->B = B; t->Hq = Hq; t->Hkv = Hkv; t->d = d; t->dtype = dtype; t->page_size = page_size;
  t->max_pages = max_pages; t->max_drafts = max_drafts;
  t->T = T; t->n_tokens = tokens; t->n_blocks = blocks;
  t->kv_bytes = (uint64_t)read * Hkv * 2 * fd::cache_row_bytes(dtype, d);
  fd::TreeParams& p = t->params;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.G = G;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)d));
  p.box_rows = page_size ? std::min(fd::kTreeTile, page_size) : fd::kTreeTile;
  p.q_tiles = rows > fd::kTreeTile ? 2 : 1;
  p.rec_rows = fd::kTreeTile * p.q_tiles;
  p.whole_items = longest <= fd::kTreeWholeTiles && all_items <= std::min(num_sms, fd::kTreeMaxCtas);
  if (p.whole_items) tiles = all_items;
  p.ctas = (int)std::min<int64_t>({tiles, (int64_t)num_sms, (int64_t)fd::kTreeMaxCtas});
  p.item_units = p.ctas ? (int)std::clamp<int64_t>(tiles * 3 / 4 / p.ctas, fd::kTreeMinItemUnits, fd::kTreeMaxItemUnits) : 0;
  const int64_t units = p.whole_items ? all_items : tiles + all_items * p.item_units;
  if (p.ctas) {
    p.run_len = (int32_t)(units / p.ctas);
    p.run_extra = (int32_t)(units % p.ctas);
  }
  int32_t cu = 0, unit = 0, cta = 1;
  int64_t base = 0;
  for (int b = 0; b < B; ++b) {
    p.cu_q[b] = cu;
    p.len[b] = seqlens[b];
    p.base[b] = (int32_t)base;
    p.unit_base[b] = unit;
    cu += drafts[b];
    base += four ? ((int64_t)seqlens[b] + fd::kBlockTokens - 1) / fd::kBlockTokens * fd::kBlockTokens : seqlens[b];
    if (!drafts[b]) continue;
    // The runs that begin behind an item's first tile: the first of them combines the item's records.
    const int items = Hkv * fd::tree_groups(drafts[b] * G), per = fd::tree_item_units(p, fd::tree_tiles(seqlens[b]));
    int last = -1;
    for (; cta < p.ctas && fd::tree_run_begin(p, cta) < unit + items * per; ++cta) {
      const int at = fd::tree_run_begin(p, cta) - unit, item = at / per;
      if (p.whole_items || at - item * per <= p.item_units || item == last) continue;
      p.split[t->splits++] = (uint16_t)cta;
      last = item;
    }
    unit += items * per;
  }
  p.cu_q[B] = cu;
  p.unit_base[B] = unit;
  t->sums_at = t->splits ? sizeof(float) * 2 * p.ctas * (size_t)fd::tree_record_floats(d, p.rec_rows) : 0;
  // A portion has no more tiles than its sequence, nor than a run has units; a group takes each (two row tiles), or every
  // other one.
  const bool two_parts = dtype == FD_BF16;
  for (int b = 0; b < B && !p.whole_items; ++b) {
    const int tiles_here = std::min(fd::tree_tiles(seqlens[b]), p.run_len + 1);
    const int jobs = drafts[b] * G > fd::kTreeTile ? tiles_here : (tiles_here + 1) / 2;
    if (drafts[b] && jobs > fd::tree_sum_tiles(two_parts)) t->long_runs = true;
  }
  t->ws_bytes = t->sums_at + (t->long_runs ? sizeof(float) * 2 * p.ctas * (size_t)d * fd::kTreeTile : 0);
  *out_tree = t;
  return FD_OK;
}

int fd_tree_destroy(fd_tree_t tree) {
  delete tree;
  return FD_OK;
}

int fd_tree_test_skip_loads(fd_tree_t t) {
  if (!t) return FD_ERR_INVALID;
  t->params.test_skip_loads = 1;
  return FD_OK;
}

int fd_tree_get_info(fd_tree_t t, fd_tree_info* info) {
  if (!t || !info) return FD_ERR_INVALID;
  info->tokens = t->T;
  info->max_drafts = t->max_drafts;
  info->ctas = t->params.ctas;
  info->workspace_bytes = t->ws_bytes;
  info->kv_bytes = t->kv_bytes;
  return FD_OK;
}

int fd_tree_decode(fd_tree_t t, const void* q, const void* k, const void* v, int num_pages, const int32_t* block_table,
                   int bt_stride, const uint64_t* mask, void* out, float* lse, void* workspace, uint32_t* status,
                   cudaStream_t stream) {
  if (!t) return FD_ERR_INVALID;
  if (t->T == 0) return FD_OK;
  if (!q || !k || !v || !out || (t->ws_bytes && !workspace)) return FD_ERR_INVALID;
  for (const void* p : {q, k, v, (const void*)out, (const void*)lse, (const void*)workspace})
    if (!fd::aligned(p, 16)) return FD_ERR_ALIGN;
  if (!fd::aligned(mask, 8) || !fd::aligned(block_table, 4) || !fd::aligned(status, 4)) return FD_ERR_ALIGN;
  fd::TreeParams p = t->params;  // per-call copy: the handle stays immutable
  int rc = fd::check_pages(t, num_pages, block_table, bt_stride, &p.page_shift);
  if (rc != FD_OK) return rc;
  const int64_t rows = t->T * t->Hq;
  const fd::Span outs[] = {fd::span(out, 2 * rows * t->d), fd::span(lse, 4 * rows),
                           fd::span(workspace, (int64_t)t->ws_bytes), fd::span(status, 4)};
  const fd::Span ins[] = {fd::span(q, 2 * rows * t->d), fd::cache_span(t, k, num_pages), fd::cache_span(t, v, num_pages),
                          fd::span(mask, 8 * t->T), fd::table_span(t, block_table, bt_stride)};
  if (fd::any_overlap(outs, ins)) return FD_ERR_INVALID;
  rc = fd::encode_cache(&p.tm_k, t, k, num_pages);
  if (rc == FD_OK) rc = fd::encode_cache(&p.tm_v, t, v, num_pages);
  if (rc != FD_OK) return rc;
  p.q = q; p.mask = mask; p.out = out; p.lse = lse; p.status = status;
  p.part = static_cast<float*>(workspace);
  p.sums = t->long_runs ? p.part + t->sums_at / sizeof(float) : nullptr;
  p.block_table = block_table; p.bt_stride = bt_stride; p.num_pages = num_pages;
  const int kind = fd::kv_kind(t->dtype);
  const bool bf16 = fd::is_bf16(t->dtype);
  const cudaError_t err = kind == fd::kKv16     ? fd::launch_tree_16(p, bf16, t->d, t->splits, stream)
                          : kind == fd::kKvE4m3 ? fd::launch_tree_8(p, t->d, t->splits, stream)
                                                : fd::launch_tree_4(p, bf16, t->d, t->splits, stream);
  if (err != cudaSuccess) {
    cudaGetLastError();
    return FD_ERR_CUDA;
  }
  return FD_OK;
}

int fd_tree_verify(fd_tree_t t, const float* target, int64_t target_stride, const float* draft, int64_t draft_stride,
                   int vocab, const int32_t* tokens, const int32_t* parents, const float* uniform, int32_t* path,
                   int32_t* emitted, int32_t* count, cudaStream_t stream) {
  if (!t || !count || vocab < 1) return FD_ERR_INVALID;
  if (t->T && (!target || !tokens || !uniform || !path || !emitted)) return FD_ERR_INVALID;
  if (vocab > FD_MAX_VOCAB || (draft && parents)) return FD_ERR_UNSUPPORTED;
  if (t->T && (target_stride < vocab || (draft && draft_stride < vocab))) return FD_ERR_INVALID;
  for (const void* p : {(const void*)target, (const void*)draft, (const void*)tokens, (const void*)parents,
                        (const void*)uniform, (const void*)path, (const void*)emitted, (const void*)count})
    if (!fd::aligned(p, 4)) return FD_ERR_ALIGN;
  const int64_t T = t->T, said = 4 * (int64_t)t->B * t->max_drafts;
  const fd::Span outs[] = {fd::span(path, said), fd::span(emitted, said), fd::span(count, 4 * (int64_t)t->B)};
  const fd::Span ins[] = {fd::span(T ? target : nullptr, 4 * ((T - 1) * target_stride + vocab)),
                          fd::span(T ? draft : nullptr, 4 * ((T - 1) * draft_stride + vocab)), fd::span(tokens, 4 * T),
                          fd::span(parents, 4 * T), fd::span(uniform, 4 * T)};
  if (fd::any_overlap(outs, ins)) return FD_ERR_INVALID;
  fd::VerifyParams p;
  p.target = target; p.draft = draft;
  p.target_stride = target_stride; p.draft_stride = draft_stride;
  p.tokens = tokens; p.parents = parents; p.uniform = uniform;
  p.path = path; p.emitted = emitted; p.count = count;
  p.vocab = vocab;
  p.max_drafts = t->max_drafts;
  std::memcpy(p.cu, t->params.cu_q, sizeof(p.cu));
  return fd::launch(reinterpret_cast<const void*>(&fd::fd_verify_kernel), dim3(t->B * fd::kVerifyCluster),
                    fd::kVerifyThreads, &p, stream);
}

int fd_tree_keep(fd_tree_t t, void* k_cache, void* v_cache, int num_pages, const int32_t* block_table, int bt_stride,
                 const int32_t* path, int path_stride, const int32_t* count, uint32_t* status, cudaStream_t stream) {
  if (!t) return FD_ERR_INVALID;
  if (t->T == 0) return FD_OK;
  if (!k_cache || !v_cache || !path || !count || path_stride < t->max_drafts) return FD_ERR_INVALID;
  if (!fd::aligned(k_cache, 16) || !fd::aligned(v_cache, 16)) return FD_ERR_ALIGN;
  if (!fd::aligned(path, 4) || !fd::aligned(count, 4) || !fd::aligned(block_table, 4) || !fd::aligned(status, 4))
    return FD_ERR_ALIGN;
  fd::KeepParams p;
  int rc = fd::check_pages(t, num_pages, block_table, bt_stride, &p.page_shift);
  if (rc != FD_OK) return rc;
  const fd::Span outs[] = {fd::cache_span(t, k_cache, num_pages), fd::cache_span(t, v_cache, num_pages),
                           fd::span(status, 4)};
  const fd::Span ins[] = {fd::span(path, 4 * ((int64_t)(t->B - 1) * path_stride + t->max_drafts)),
                          fd::span(count, 4 * (int64_t)t->B), fd::table_span(t, block_table, bt_stride)};
  if (fd::any_overlap(outs, ins)) return FD_ERR_INVALID;
  p.k_cache = static_cast<uint8_t*>(k_cache); p.v_cache = static_cast<uint8_t*>(v_cache);
  p.block_table = block_table; p.path = path; p.count = count; p.status = status;
  p.Hkv = t->Hkv; p.d = t->d; p.num_pages = num_pages; p.bt_stride = bt_stride; p.path_stride = path_stride;
  const int kind = fd::kv_kind(t->dtype);
  p.pieces = kind == fd::kKvE2m1 ? t->Hkv * (t->d / 8 + t->d / 16)
                                 : (int)(t->Hkv * fd::cache_row_bytes(t->dtype, t->d) / 16);
  std::memcpy(p.cu, t->params.cu_q, sizeof(p.cu));
  std::memcpy(p.base, t->params.base, sizeof(p.base));
  for (int b = 0; b < t->B; ++b) p.first[b] = t->params.len[b] - (p.cu[b + 1] - p.cu[b]);
  const dim3 grid(2 * ((p.pieces + fd::kKeepThreads - 1) / fd::kKeepThreads), t->B);
  const void* fn = kind == fd::kKv16     ? reinterpret_cast<const void*>(&fd::fd_keep_kernel<fd::kKv16>)
                   : kind == fd::kKvE4m3 ? reinterpret_cast<const void*>(&fd::fd_keep_kernel<fd::kKvE4m3>)
                                         : reinterpret_cast<const void*>(&fd::fd_keep_kernel<fd::kKvE2m1>);
  return fd::launch(fn, grid, fd::kKeepThreads, &p, stream);
}

}  // extern "C"
