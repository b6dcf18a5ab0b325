// Internal launchers of the prompt operators (lin_prompt.h).
#pragma once

#include "internal.h"
#include "lin_prompt.h"

namespace lin {

// kv_plan.cu
cudaError_t launch_kv_plan(const lin_kv_plan_args_t& a, cudaStream_t stream);

// rope.cu
cudaError_t launch_rope(const lin_kv_cache_t* cache, const lin_rope_args_t& a, cudaStream_t stream);

// chunk_attn.cu
size_t chunk_need(const lin_kv_cache_t& cache, const lin_attn_chunk_args_t& a);
size_t chunk_workspace(const lin_kv_cache_t& cache, const lin_attn_chunk_args_t& a);
cudaError_t launch_attn_chunk(const lin_kv_cache_t& cache, const lin_attn_chunk_args_t& a, void* workspace,
                              cudaStream_t stream);

}  // namespace lin
