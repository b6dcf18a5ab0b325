// Decode attention kernels for heads of 256 channels (attn_kernel.cuh).

#include "attn_kernel.cuh"

namespace lin {
namespace attn {

cudaError_t launch_d256(const Plan& p, int row_tiles, int grid, cudaStream_t s) {
  return p.c.dtype == LIN_BF16 ? launch_rows<256, LIN_BF16>(p, row_tiles, grid, s)
                               : launch_rows<256, LIN_F32>(p, row_tiles, grid, s);
}

}  // namespace attn
}  // namespace lin
