// Tensor-memory decode attention kernels for heads of 128 channels (attn_umma.cuh).

#include "attn_umma.cuh"

namespace lin {
namespace attn {

cudaError_t launch_umma_d128(const Plan& p, int grid, cudaStream_t s) { return launch_umma_rows<128>(p, grid, s); }

}  // namespace attn
}  // namespace lin
