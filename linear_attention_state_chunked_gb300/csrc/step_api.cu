// C-ABI entry points of lin_step.h. One translation unit with api.cu: the
// checks here share its helpers and the thread's last-error text, which are
// file-local there.

#include "api.cu"
#include "step_internal.h"

namespace {

int check_cache(const lin_kv_cache_t* c) {
  if (!c) return fail(LIN_EINVAL, "cache is NULL");
  if (c->num_layers <= 0 || c->num_pages <= 0 || c->page_size <= 0 || c->num_kv_heads <= 0)
    return fail(LIN_EINVAL, "cache: num_layers, num_pages, page_size, num_kv_heads must be positive");
  if (!valid_dtype(c->dtype)) return fail(LIN_EINVAL, "cache: dtype must be LIN_F32 or LIN_BF16");
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(LIN_EUNSUPPORTED, "cache: head_dim must be 64, 128 or 256 (got %d)", c->head_dim);
  if (!c->k || !c->v) return fail(LIN_EINVAL, "cache: k / v is NULL");
  if (!aligned16(c->k) || !aligned16(c->v)) return fail(LIN_EINVAL, "cache: k / v must be 16-byte aligned");
  // the four axes nest in some order: sorted by stride, each stride covers
  // the extent of the axes below it (the stride of an axis of one is not used)
  int64_t stride[4] = {c->head_stride, c->token_stride, c->page_stride, c->layer_stride};
  int64_t count[4] = {c->num_kv_heads, c->page_size, c->num_pages, c->num_layers};
  for (int i = 0; i < 4; ++i)
    if (count[i] > 1 && (stride[i] < 0 || (stride[i] & 15)))
      return fail(LIN_EINVAL, "cache: strides must be non-negative multiples of 16 bytes");
  for (int i = 1; i < 4; ++i)
    for (int j = i; j > 0 && stride[j] < stride[j - 1]; --j) {
      const int64_t s = stride[j], n = count[j];
      stride[j] = stride[j - 1], count[j] = count[j - 1];
      stride[j - 1] = s, count[j - 1] = n;
    }
  int64_t extent = int64_t(c->head_dim) * lin::dtype_size(c->dtype);
  for (int i = 0; i < 4; ++i) {
    if (count[i] == 1) continue;
    if (stride[i] < extent) return fail(LIN_EINVAL, "cache: strides make rows overlap");
    if (stride[i] > INT64_MAX / count[i]) return fail(LIN_EINVAL, "cache: strides out of range");
    extent = stride[i] * (count[i] - 1) + extent;
  }
  return LIN_OK;
}

// Rows of `heads` head vectors, `tokens` to a request. The stride of a single
// token or request is not used.
int check_rows(const char* what, int64_t req_stride, int64_t token_stride, int64_t row_bytes,
               int batch, int tokens) {
  if ((tokens > 1 && (token_stride < 0 || (token_stride & 15))) ||
      (batch > 1 && (req_stride < 0 || (req_stride & 15))))
    return fail(LIN_EINVAL, "%s: strides must be non-negative multiples of 16 bytes", what);
  if ((tokens > 1 && token_stride < row_bytes) || (batch > 1 && req_stride < row_bytes))
    return fail(LIN_EINVAL, "%s: strides smaller than one row of %lld bytes", what,
                static_cast<long long>(row_bytes));
  return LIN_OK;
}

int check_attn(const lin_kv_cache_t* c, const lin_attn_args_t* a) {
  int rc = check_cache(c);
  if (rc) return rc;
  if (!a) return fail(LIN_EINVAL, "attn args is NULL");
  if (a->layer < 0 || a->layer >= c->num_layers)
    return fail(LIN_EINVAL, "attn: layer %d outside [0, %d)", a->layer, c->num_layers);
  if (a->batch < 0 || a->batch > 65535) return fail(LIN_EINVAL, "attn: batch outside [0, 65535]");
  if (a->n_q < 1) return fail(LIN_EINVAL, "attn: n_q must be >= 1");
  if (a->n_q > lin::kAttnMaxQuery)
    return fail(LIN_EUNSUPPORTED, "attn: at most %d query tokens, not %d", lin::kAttnMaxQuery, a->n_q);
  if (a->num_q_heads < 1 || a->num_q_heads % c->num_kv_heads)
    return fail(LIN_EINVAL, "attn: num_q_heads %d is no multiple of num_kv_heads %d", a->num_q_heads,
                c->num_kv_heads);
  if (a->num_q_heads > 65536) return fail(LIN_EUNSUPPORTED, "attn: num_q_heads above 65536");
  if (!valid_dtype(a->out_dtype)) return fail(LIN_EINVAL, "attn: out_dtype");
  if (a->max_pages < 0) return fail(LIN_EINVAL, "attn: negative max_pages");
  return LIN_OK;
}

}  // namespace

extern "C" {

int lin_state_kv_append(const lin_kv_cache_t* c, const lin_kv_append_args_t* a, void* stream) {
  int rc = check_cache(c);
  if (rc) return rc;
  if (!a) return fail(LIN_EINVAL, "append args is NULL");
  if (a->layer < 0 || a->layer >= c->num_layers)
    return fail(LIN_EINVAL, "append: layer %d outside [0, %d)", a->layer, c->num_layers);
  if (a->batch < 0 || a->n < 0 || a->max_pages < 0)
    return fail(LIN_EINVAL, "append: negative batch / n / max_pages");
  if (a->batch == 0 || a->n == 0) return ok();
  if (!a->k || !a->v || !a->pos || (a->max_pages > 0 && !a->page_table))
    return fail(LIN_EINVAL, "append: k / v / page_table / pos is NULL");
  if (!aligned16(a->k) || !aligned16(a->v)) return fail(LIN_EINVAL, "append: k and v must be 16-byte aligned");
  if (!a->parent != !a->accept_node)
    return fail(LIN_EINVAL, "append: a draft tree needs both parent and accept_node");
  if (a->parent && a->n_tok) return fail(LIN_EINVAL, "append: n_tok and a draft tree exclude each other");
  if (a->parent && a->n > 32)
    return fail(LIN_EUNSUPPORTED, "append: a draft tree holds at most 32 drafts, not %d", a->n);
  rc = check_rows("append: k / v", a->req_stride, a->token_stride,
                  int64_t(c->num_kv_heads) * c->head_dim * lin::dtype_size(c->dtype), a->batch, a->n);
  if (rc) return rc;
  if (a->page_table_stride < a->max_pages && a->batch > 1)
    return fail(LIN_EINVAL, "append: page_table_stride smaller than max_pages");
  cudaError_t e = lin::launch_kv_append(*c, *a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "lin_state_kv_append launch");
  return ok();
}

size_t lin_state_attn_workspace(const lin_kv_cache_t* c, const lin_attn_args_t* a) {
  if (check_attn(c, a) || a->batch == 0) return 0;
  return lin::attn_workspace(*c, *a);
}

int lin_state_attn_decode(const lin_kv_cache_t* c, const lin_attn_args_t* a, void* workspace,
                          size_t workspace_bytes, void* stream) {
  int rc = check_attn(c, a);
  if (rc) return rc;
  if (a->batch == 0) return ok();
  if (!a->q || !a->out || !a->kv_len || (a->max_pages > 0 && !a->page_table))
    return fail(LIN_EINVAL, "attn: q / out / page_table / kv_len is NULL");
  if (!aligned16(a->q) || !aligned16(a->out)) return fail(LIN_EINVAL, "attn: q and out must be 16-byte aligned");
  rc = check_rows("attn: q", a->req_stride, a->token_stride,
                  int64_t(a->num_q_heads) * c->head_dim * lin::dtype_size(c->dtype), a->batch, a->n_q);
  if (rc) return rc;
  if (a->page_table_stride < a->max_pages && a->batch > 1)
    return fail(LIN_EINVAL, "attn: page_table_stride smaller than max_pages");
  const size_t need = lin::attn_need(*c, *a);
  if (workspace_bytes < need || (need > 0 && !workspace))
    return fail(LIN_EWORKSPACE, "attn: workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  if (!aligned16(workspace)) return fail(LIN_EINVAL, "attn: workspace must be 16-byte aligned");
  cudaError_t e = lin::launch_attn_decode(*c, *a, workspace, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "lin_state_attn_decode launch");
  return ok();
}

int lin_state_block_norm(const lin_norm_args_t* a, void* stream) {
  if (!a) return fail(LIN_EINVAL, "norm args is NULL");
  if (a->rows < 0 || a->channels < 1) return fail(LIN_EINVAL, "norm: rows / channels");
  if (a->channels > lin::kNormMaxChannels)
    return fail(LIN_EUNSUPPORTED, "norm: at most %d channels, not %d", lin::kNormMaxChannels, a->channels);
  if (!valid_dtype(a->x_dtype) || !valid_dtype(a->io_dtype) || !valid_dtype(a->h_dtype))
    return fail(LIN_EINVAL, "norm: x_dtype / io_dtype / h_dtype");
  if (a->rows == 0) return ok();
  if (a->rows > INT32_MAX) return fail(LIN_EUNSUPPORTED, "norm: more than 2^31 - 1 rows");
  if (!a->x || (!a->h_out && !a->y)) return fail(LIN_EINVAL, "norm: x is NULL, or both h_out and y are");
  if (!a->w_pre != !a->y) return fail(LIN_EINVAL, "norm: w_pre and y go together");
  if (a->w_post && (a->group < 1 || a->channels % a->group))
    return fail(LIN_EINVAL, "norm: group %d does not divide channels %d", a->group, a->channels);
  if (a->gate ? (a->gate_act != LIN_ACT_SILU && a->gate_act != LIN_ACT_SIGMOID) : a->gate_act != LIN_ACT_NONE)
    return fail(LIN_EINVAL, "norm: gate_act");
  const struct { const void* p; int64_t s; int dt; const char* what; } rows[5] = {
      {a->x, a->x_stride, a->x_dtype, "x"}, {a->gate, a->gate_stride, a->io_dtype, "gate"},
      {a->residual, a->residual_stride, a->h_dtype, "residual"}, {a->h_out, a->h_stride, a->h_dtype, "h_out"},
      {a->y, a->y_stride, a->io_dtype, "y"}};
  for (const auto& r : rows) {
    if (!r.p) continue;
    if (a->rows > 1 && r.s < a->channels) return fail(LIN_EINVAL, "norm: %s: row stride smaller than a row", r.what);
    if (reinterpret_cast<uintptr_t>(r.p) % lin::dtype_size(r.dt))
      return fail(LIN_EINVAL, "norm: %s is not aligned to its type", r.what);
  }
  const void* weights[3] = {a->w_post, a->scale_w, a->w_pre};
  for (const void* w : weights)
    if (w && reinterpret_cast<uintptr_t>(w) % lin::dtype_size(a->io_dtype))
      return fail(LIN_EINVAL, "norm: a weight is not aligned to its type");
  cudaError_t e = lin::launch_block_norm(*a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "lin_state_block_norm launch");
  return ok();
}

}  // extern "C"
