// Tree attention over 16-bit caches.
#include "fd_tree_attn.cuh"

namespace fd {
cudaError_t launch_tree_16(const TreeParams& p, bool bf16, int d, int splits, cudaStream_t s) {
  if (bf16)
    return d == 64 ? tree::launch<__nv_bfloat16, 64, kKv16>(p, splits, s) : tree::launch<__nv_bfloat16, 128, kKv16>(p, splits, s);
  return d == 64 ? tree::launch<__half, 64, kKv16>(p, splits, s) : tree::launch<__half, 128, kKv16>(p, splits, s);
}
}  // namespace fd
