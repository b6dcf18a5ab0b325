// Tensor-memory chunk attention kernels for heads of 256 channels (chunk_umma.cuh).

#include "chunk_umma.cuh"

namespace lin {
namespace chunk {

cudaError_t launch_umma_d256(const Plan& p, const Maps& m, cudaStream_t s) {
  return launch_umma_tiles<256>(p, m, s);
}

}  // namespace chunk
}  // namespace lin
