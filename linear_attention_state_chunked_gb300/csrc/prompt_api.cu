// C-ABI entry points of lin_prompt.h. One translation unit with step_api.cu and api.cu:
// the checks here share their helpers and the thread's last-error text, which are
// file-local there.

#include "step_api.cu"
#include "prompt_internal.h"

namespace {

int check_chunk(const lin_kv_cache_t* c, const lin_attn_chunk_args_t* a) {
  int rc = check_cache(c);
  if (rc) return rc;
  if (!a) return fail(LIN_EINVAL, "chunk args is NULL");
  if (a->layer < 0 || a->layer >= c->num_layers)
    return fail(LIN_EINVAL, "chunk: layer %d outside [0, %d)", a->layer, c->num_layers);
  if (a->batch < 0 || a->batch > 65535) return fail(LIN_EINVAL, "chunk: batch outside [0, 65535]");
  if (a->tokens < 0) return fail(LIN_EINVAL, "chunk: negative tokens");
  if (a->num_q_heads < 1 || a->num_q_heads % c->num_kv_heads)
    return fail(LIN_EINVAL, "chunk: num_q_heads %d is no multiple of num_kv_heads %d", a->num_q_heads,
                c->num_kv_heads);
  if (a->num_q_heads > 65536) return fail(LIN_EUNSUPPORTED, "chunk: num_q_heads above 65536");
  if (!valid_dtype(a->out_dtype)) return fail(LIN_EINVAL, "chunk: out_dtype");
  if (a->max_pages < 0) return fail(LIN_EINVAL, "chunk: negative max_pages");
  return LIN_OK;
}

// A row of head vectors per token, 16-byte aligned.
int check_packed(const char* what, const void* p, int64_t stride, int64_t row_bytes, int tokens) {
  if (!aligned16(p)) return fail(LIN_EINVAL, "%s must be 16-byte aligned", what);
  if (tokens > 1 && (stride < row_bytes || (stride & 15)))
    return fail(LIN_EINVAL, "%s: token stride must be a multiple of 16 bytes, one row of %lld at least", what,
                static_cast<long long>(row_bytes));
  return LIN_OK;
}

}  // namespace

extern "C" {

int lin_state_kv_plan(const lin_kv_plan_args_t* a, void* stream) {
  if (!a) return fail(LIN_EINVAL, "plan args is NULL");
  if (a->batch < 0 || a->tokens < 0 || a->max_pages < 0 || a->num_free < 0)
    return fail(LIN_EINVAL, "plan: negative batch / tokens / max_pages / num_free");
  if (a->batch > 1 << 30) return fail(LIN_EUNSUPPORTED, "plan: batch above 2^30");
  if (a->page_size < 1 || a->num_pages < 1) return fail(LIN_EINVAL, "plan: page_size and num_pages must be positive");
  if (!a->n_new && a->n < 0) return fail(LIN_EINVAL, "plan: negative n");
  if (a->parent && a->n_new) return fail(LIN_EINVAL, "plan: n_new and a draft tree exclude each other");
  if (a->parent && a->n > 32)
    return fail(LIN_EUNSUPPORTED, "plan: a draft tree holds at most 32 drafts, not %d", a->n);
  if (a->batch > 0 && (!a->length || (a->max_pages > 0 && !a->page_table)))
    return fail(LIN_EINVAL, "plan: length / page_table is NULL");
  if (a->page_table_stride < a->max_pages && a->batch > 1)
    return fail(LIN_EINVAL, "plan: page_table_stride smaller than max_pages");
  if (a->kv_len && (a->kv_len == a->length || a->kv_len == a->n_new))
    return fail(LIN_EINVAL, "plan: kv_len must not be an input, which is read while it is written");
  cudaError_t e = lin::launch_kv_plan(*a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "lin_state_kv_plan launch");
  return ok();
}

int lin_state_rope(const lin_kv_cache_t* c, const lin_rope_args_t* a, void* stream) {
  if (c) {
    int rc = check_cache(c);
    if (rc) return rc;
  }
  if (!a) return fail(LIN_EINVAL, "rope args is NULL");
  if (a->tokens < 0 || a->num_q_heads < 0 || a->num_k_heads < 0)
    return fail(LIN_EINVAL, "rope: negative tokens / num_q_heads / num_k_heads");
  if (!valid_dtype(a->dtype)) return fail(LIN_EINVAL, "rope: dtype must be LIN_F32 or LIN_BF16");
  if (a->head_dim < 8 || a->head_dim > 256 || a->head_dim % 8)
    return fail(LIN_EUNSUPPORTED, "rope: head_dim must be a multiple of 8 up to 256 (got %d)", a->head_dim);
  if (a->rot_dim < 2 || a->rot_dim > a->head_dim || a->rot_dim % 2)
    return fail(LIN_EINVAL, "rope: rot_dim must be even, 2 to head_dim (got %d)", a->rot_dim);
  if (a->num_q_heads > 65536 || a->num_k_heads > 65536)
    return fail(LIN_EUNSUPPORTED, "rope: num_q_heads / num_k_heads above 65536");
  if (c) {
    if (a->layer < 0 || a->layer >= c->num_layers)
      return fail(LIN_EINVAL, "rope: layer %d outside [0, %d)", a->layer, c->num_layers);
    if (c->num_kv_heads != a->num_k_heads || c->head_dim != a->head_dim || c->dtype != a->dtype)
      return fail(LIN_EINVAL, "rope: the cache has other heads, head_dim or dtype than k");
  }
  const bool q = a->q_out && a->num_q_heads > 0, k = (a->k_out || c) && a->num_k_heads > 0;
  if (!q && !k) return fail(LIN_EINVAL, "rope: nothing to write: no q_out, k_out or cache");
  if (a->tokens == 0) return ok();
  if (!a->position || !a->inv_freq || (q && !a->q) || (k && !a->k) || (c && (!a->v || !a->slot)))
    return fail(LIN_EINVAL, "rope: position / inv_freq / q / k / v / slot is NULL");
  const int64_t head = int64_t(a->head_dim) * lin::dtype_size(a->dtype);
  const struct { bool used; const void* p; int64_t s; int heads; const char* what; } rows[5] = {
      {q, a->q, a->q_stride, a->num_q_heads, "rope: q"},
      {q, a->q_out, a->q_out_stride, a->num_q_heads, "rope: q_out"},
      {k, a->k, a->k_stride, a->num_k_heads, "rope: k"},
      {k && a->k_out, a->k_out, a->k_out_stride, a->num_k_heads, "rope: k_out"},
      {c != nullptr, a->v, a->v_stride, a->num_k_heads, "rope: v"}};
  for (const auto& r : rows) {
    if (!r.used) continue;
    int rc = check_packed(r.what, r.p, r.s, r.heads * head, a->tokens);
    if (rc) return rc;
  }
  if ((q && a->q_out == a->q && a->q_out_stride != a->q_stride && a->tokens > 1) ||
      (k && a->k_out == a->k && a->k_out_stride != a->k_stride && a->tokens > 1))
    return fail(LIN_EINVAL, "rope: an output in its input's place must have its stride");
  cudaError_t e = lin::launch_rope(c, *a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "lin_state_rope launch");
  return ok();
}

size_t lin_state_attn_chunk_workspace(const lin_kv_cache_t* c, const lin_attn_chunk_args_t* a) {
  if (check_chunk(c, a) || a->batch == 0 || a->tokens == 0) return 0;
  return lin::chunk_workspace(*c, *a);
}

int lin_state_attn_chunk(const lin_kv_cache_t* c, const lin_attn_chunk_args_t* a, void* workspace,
                         size_t workspace_bytes, void* stream) {
  int rc = check_chunk(c, a);
  if (rc) return rc;
  if (a->batch == 0 || a->tokens == 0) return ok();
  if (!a->q || !a->out || !a->kv_len || !a->cu_seqlens || (a->max_pages > 0 && !a->page_table))
    return fail(LIN_EINVAL, "chunk: q / out / page_table / cu_seqlens / kv_len is NULL");
  if (!aligned16(a->out)) return fail(LIN_EINVAL, "chunk: out must be 16-byte aligned");
  rc = check_packed("chunk: q", a->q, a->token_stride,
                    int64_t(a->num_q_heads) * c->head_dim * lin::dtype_size(c->dtype), a->tokens);
  if (rc) return rc;
  if (a->page_table_stride < a->max_pages && a->batch > 1)
    return fail(LIN_EINVAL, "chunk: page_table_stride smaller than max_pages");
  const size_t need = lin::chunk_need(*c, *a);
  if (workspace_bytes < need || !workspace)
    return fail(LIN_EWORKSPACE, "chunk: workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  if (!aligned16(workspace)) return fail(LIN_EINVAL, "chunk: workspace must be 16-byte aligned");
  cudaError_t e = lin::launch_attn_chunk(*c, *a, workspace, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "lin_state_attn_chunk launch");
  return ok();
}

}  // extern "C"
