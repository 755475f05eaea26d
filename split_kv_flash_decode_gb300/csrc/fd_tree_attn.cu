// Attention of drafted tokens over the cache (fd_tree_decode).  See fd.h for the contract.
#include "fd_kernel.cuh"
#include "fd_tree.h"

namespace fd {
namespace {

// Element e of row `row` (tokens) of KV head h.
template <typename T, int D, int KV>
__device__ __forceinline__ float element(const void* cache, int64_t row, int h, int H, int e, bool is_v) {
  if constexpr (KV == kKv16) {
    return static_cast<float>(reinterpret_cast<const T*>(cache)[(row * H + h) * D + e]);
  } else if constexpr (KV == kKvE4m3) {
    const uint32_t x = reinterpret_cast<const uint8_t*>(cache)[(row * H + h) * D + e];
    return dev::Elem<__half>::to_f2(dev::e4m3x2_to_f16x2(x)).x;
  } else {
    const uint8_t* blk = reinterpret_cast<const uint8_t*>(cache) + ((row >> kBlockShift) * H + h) * (9 * D);
    const int r = (int)(row & (kBlockTokens - 1));
    const int g = e / (D / 8), swap = ((D == 128 ? g : g >> 1) & 1) << 2;
    const int at = is_v ? g * D + ((r >> 1) ^ swap) * (D / 8) + (r & 1) * (D / 16) + (e % (D / 8)) / 2 : r * (D / 2) + e / 2;
    const uint32_t code = blk[at] >> (4 * (e & 1)) & 15u;
    uint32_t f[4];
    dev::e2m1x8_to_f16x8(code, f);
    const uint32_t s = blk[8 * D + (is_v ? 16 * (e / 16) + r : r * (D / 16) + e / 16)];
    return dev::Elem<__half>::to_f2(f[0]).x * dev::Elem<__half>::to_f2(dev::e4m3x2_to_f16x2(s)).x;
  }
}

// One CTA: one query row.
template <typename T, int D, int KV>
__global__ void __launch_bounds__(128) fd_tree_kernel(const __grid_constant__ TreeParams p) {
  __shared__ float qs[D], ps[128], red[4];
  dev::pdl_launch_dependents();
  dev::pdl_wait();
  const int t = blockIdx.x / p.Hq, h = blockIdx.x - t * p.Hq, kvh = h / (p.Hq / p.Hkv), tid = threadIdx.x;
  int b = 0;
  while (p.cu_q[b + 1] <= t) ++b;
  const int n = p.cu_q[b + 1] - p.cu_q[b], i = t - p.cu_q[b], L = p.len[b];
  const uint64_t mask = p.mask != nullptr ? p.mask[t] : ~0ull >> (63 - i);
  auto row_of = [&](int r) {
    if (p.block_table == nullptr) return (int64_t)p.base[b] + r;
    const int pg = p.block_table[(int64_t)b * p.bt_stride + (r >> p.page_shift)];
    return (uint32_t)pg >= (uint32_t)p.num_pages ? (int64_t)-1 : ((int64_t)pg << p.page_shift) + (r & ((1 << p.page_shift) - 1));
  };
  for (int e = tid; e < D; e += 128) qs[e] = static_cast<float>(reinterpret_cast<const T*>(p.q)[((int64_t)t * p.Hq + h) * D + e]);
  __syncthreads();
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int j0 = 0; j0 < L; j0 += 128) {
    const int j = j0 + tid, node = j - (L - n);
    float s = -INFINITY;
    if (j < L && (node < 0 || (mask >> node & 1))) {
      const int64_t row = row_of(j);
      s = 0.f;
      if (row >= 0)
        for (int e = 0; e < D; ++e) s = fmaf(qs[e], element<T, D, KV>(p.k, row, kvh, p.Hkv, e, false), s);
      s *= p.scale_log2;
    }
    float mx = s;
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float mn = fmaxf(m, mx), c = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float pr = s == -INFINITY ? 0.f : exp2f(s - mn);
    ps[tid] = pr;
    float sum = pr;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    l = l * c + red[0] + red[1] + red[2] + red[3];
    acc *= c;
    m = mn;
    if (tid < D)
      for (int k = 0; k < 128 && j0 + k < L; ++k) {
        const int64_t row = ps[k] != 0.f ? row_of(j0 + k) : -1;
        if (row >= 0) acc = fmaf(ps[k], element<T, D, KV>(p.v, row, kvh, p.Hkv, tid, true), acc);
      }
  }
  if (tid < D)
    reinterpret_cast<T*>(p.out)[((int64_t)t * p.Hq + h) * D + tid] = dev::Elem<T>::from_f(l > 0.f ? acc / l : 0.f);
  if (tid == 0 && p.lse != nullptr) p.lse[(int64_t)t * p.Hq + h] = l > 0.f ? m * dev::kLn2 + logf(l) : -INFINITY;
}

template <typename T, int D, int KV>
cudaError_t run(const TreeParams& p, int T_, cudaStream_t s) {
  fd_tree_kernel<T, D, KV><<<T_ * p.Hq, 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree(const TreeParams& p, int dtype, int d, int T, cudaStream_t s) {
  if (d == 64) {
    if (dtype == FD_F16) return run<__half, 64, kKv16>(p, T, s);
    if (dtype == FD_BF16) return run<__nv_bfloat16, 64, kKv16>(p, T, s);
    if (dtype == FD_F16_E4M3KV) return run<__half, 64, kKvE4m3>(p, T, s);
    if (dtype == FD_F16_E2M1KV) return run<__half, 64, kKvE2m1>(p, T, s);
    return run<__nv_bfloat16, 64, kKvE2m1>(p, T, s);
  }
  if (dtype == FD_F16) return run<__half, 128, kKv16>(p, T, s);
  if (dtype == FD_BF16) return run<__nv_bfloat16, 128, kKv16>(p, T, s);
  if (dtype == FD_F16_E4M3KV) return run<__half, 128, kKvE4m3>(p, T, s);
  if (dtype == FD_F16_E2M1KV) return run<__half, 128, kKvE2m1>(p, T, s);
  return run<__nv_bfloat16, 128, kKvE2m1>(p, T, s);
}

}  // namespace fd
