// bf16 instantiations of the decode kernels over a 4-bit cache.
#include "fd_kernel.cuh"

namespace fd {
cudaError_t launch_kv4_bf16(const Params& p, int d, int G, int mode, bool pdl, int grid,
                           cudaStream_t s) {
  return launch_typed_kv4<__nv_bfloat16>(p, d, G, mode, pdl, grid, s);
}
}  // namespace fd
