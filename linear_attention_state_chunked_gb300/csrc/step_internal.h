// Internal launchers of the decode-step operators (lin_step.h).
#pragma once

#include "internal.h"
#include "lin_step.h"

namespace lin {

// kv_cache.cu
cudaError_t launch_kv_append(const lin_kv_cache_t& cache, const lin_kv_append_args_t& a,
                             cudaStream_t stream);

// attn_decode.cu
constexpr int kAttnMaxQuery = 32;
size_t attn_need(const lin_kv_cache_t& cache, const lin_attn_args_t& a);
size_t attn_workspace(const lin_kv_cache_t& cache, const lin_attn_args_t& a);
cudaError_t launch_attn_decode(const lin_kv_cache_t& cache, const lin_attn_args_t& a,
                               void* workspace, cudaStream_t stream);

// block_norm.cu
constexpr int kNormMaxChannels = 32768;
cudaError_t launch_block_norm(const lin_norm_args_t& a, cudaStream_t stream);

}  // namespace lin
