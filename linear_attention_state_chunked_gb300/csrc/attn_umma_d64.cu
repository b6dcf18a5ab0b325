// Tensor-memory decode attention kernels for heads of 64 channels (attn_umma.cuh).

#include "attn_umma.cuh"

namespace lin {
namespace attn {

cudaError_t launch_umma_d64(const Plan& p, int grid, cudaStream_t s) { return launch_umma_rows<64>(p, grid, s); }

}  // namespace attn
}  // namespace lin
