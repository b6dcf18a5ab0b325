// Warp-level MMA chunk attention kernels for heads of 64 channels (chunk_mma.cuh).

#include "chunk_mma.cuh"

namespace lin {
namespace chunk {

cudaError_t launch_mma_d64(const Plan& p, cudaStream_t s) { return launch_mma_types<64>(p, s); }

}  // namespace chunk
}  // namespace lin
