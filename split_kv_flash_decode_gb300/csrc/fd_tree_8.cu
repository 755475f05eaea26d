// Tree attention over FP8 (E4M3) caches.
#include "fd_tree_attn.cuh"

namespace fd {
cudaError_t launch_tree_8(const TreeParams& p, int d, int splits, cudaStream_t s) {
  return d == 64 ? tree::launch<__half, 64, kKvE4m3>(p, splits, s) : tree::launch<__half, 128, kKvE4m3>(p, splits, s);
}
}  // namespace fd
