// Tree attention over 4-bit caches.
#include "fd_tree_attn.cuh"

namespace fd {
cudaError_t launch_tree_4(const TreeParams& p, bool bf16, int d, int splits, cudaStream_t s) {
  if (bf16)
    return d == 64 ? tree::launch<__nv_bfloat16, 64, kKvE2m1>(p, splits, s) : tree::launch<__nv_bfloat16, 128, kKvE2m1>(p, splits, s);
  return d == 64 ? tree::launch<__half, 64, kKvE2m1>(p, splits, s) : tree::launch<__half, 128, kKvE2m1>(p, splits, s);
}
}  // namespace fd
