// Tensor-memory chunk attention kernels for heads of 64 channels (chunk_umma.cuh).

#include "chunk_umma.cuh"

namespace lin {
namespace chunk {

cudaError_t launch_umma_d64(const Plan& p, const Maps& m, cudaStream_t s) {
  return launch_umma_tiles<64>(p, m, s);
}

}  // namespace chunk
}  // namespace lin
