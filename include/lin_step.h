/*
 * lin_step.h -- the rest of a hybrid model's decode step, beside the
 * linear-attention state path of lin_state.h and under its conventions
 * (memory, streams, errors, status bits): a paged key-value cache and the
 * decode attention that reads it, for the model's full-attention layers, and
 * the norms around a block with its gate and residual.
 *
 * Every buffer is the caller's, every call only enqueues work on `stream`,
 * host-detectable errors return LIN_E* before any launch, and what only a
 * kernel can see sets LIN_ST_* bits in the optional device word `status`.
 */
#ifndef LIN_STEP_H_
#define LIN_STEP_H_

#include "lin_state.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- device status bit (with those of lin_state.h) ----------------------- */
#define LIN_ST_BAD_PAGE 512    /* a page id outside [0, num_pages) where a token lies */

/* ---- the paged key-value cache -------------------------------------------
 * k, v: bases of [num_layers][num_pages][page_size][num_kv_heads][head_dim]
 * in `dtype`; head_dim is contiguous, the other strides are given in bytes
 * (multiples of 16, the same for k and v; that of an axis of one is not looked
 * at, here and below), so tokens-first and heads-first
 * pages and views of a combined tensor all do. A request's token t lies in
 * page page_table[r][t / page_size], row t % page_size. page_size is any
 * positive number; head_dim is 64, 128 or 256 (else LIN_EUNSUPPORTED). */
typedef struct {
  int32_t num_layers, num_pages, page_size, num_kv_heads, head_dim;
  int32_t dtype; /* lin_dtype_t */
  void* k;       /* device */
  void* v;       /* device */
  int64_t layer_stride, page_stride, token_stride, head_stride;
} lin_kv_cache_t;

/* ---- append ----------------------------------------------------------------
 * Writes request r's new keys and values k, v [batch][n][num_kv_heads][head_dim]
 * (the cache's dtype; request and token strides in bytes, multiples of 16, so
 * views of a projection's output do) to the token positions from pos[r] on.
 *   no counts:   all n tokens, token j to pos[r] + j;
 *   n_tok:       the first n_tok[r] (0..n) of them: a ragged prompt, or the
 *                accepted prefix of a chain of drafts;
 *   parent, accept_node (n <= 32): the accepted path of a draft tree, as in
 *                lin_commit_args_t: the node at depth i goes to pos[r] + i;
 *                accept_node -1 writes nothing.
 * pos[r] < 0 marks padding. A position past max_pages * page_size sets
 * LIN_ST_BAD_SEQLEN, a page id outside [0, num_pages) LIN_ST_BAD_PAGE (that
 * token is left out), a count outside [0, n] LIN_ST_BAD_ACCEPT and a tree that
 * breaks its rules LIN_ST_BAD_TREE (that request is left out). Requests must
 * not share the pages that they write. */
typedef struct {
  int32_t layer, batch, n;
  int32_t max_pages;         /* page table entries per request */
  const void* k;             /* device */
  const void* v;             /* device */
  int64_t req_stride, token_stride; /* bytes, of k and v alike */
  const int32_t* page_table; /* device [batch], rows page_table_stride entries apart */
  int64_t page_table_stride;
  const int32_t* pos;        /* device [batch] */
  const int32_t* n_tok;      /* device [batch] or NULL */
  const int32_t* parent;     /* device [batch][n] or NULL */
  const int32_t* accept_node;/* device [batch], with parent */
  int32_t* status;
} lin_kv_append_args_t;

LIN_API int lin_state_kv_append(const lin_kv_cache_t* cache, const lin_kv_append_args_t* args,
                                void* stream);

/* ---- decode attention ------------------------------------------------------
 * Attention of each request's n_q newest tokens (1: a decode step; up to 32:
 * the drafts of a verify) over its cached tokens, those n_q included: append
 * them first. kv_len[r] counts them all. Query head h reads key-value head
 * h / (num_q_heads / num_kv_heads). Query j sees
 *   every token t < kv_len[r] - n_q, and of the drafts d = t - (kv_len[r] - n_q)
 *   those with d <= j (a chain), or, with `parent` (device [batch][n_q], the
 *   tree of lin_decode_args_t), j itself and its ancestors.
 * out[r][j][h] = sum_t softmax_t(scale q . k_t) v_t; a query that sees nothing
 * (kv_len 0, or kv_len < n_q) gives zeros. Keys and values that a query does
 * not see have no part in its output, whatever they hold (NaN too).
 * q [batch][n_q][num_q_heads][head_dim] has the cache's dtype, request and
 * token strides in bytes (multiples of 16); out is contiguous, in out_dtype.
 * kv_len[r] < 0 marks padding (out[r] is left as it is). A kv_len past
 * max_pages * page_size sets LIN_ST_BAD_SEQLEN, a bad tree LIN_ST_BAD_TREE
 * (request left out); a page id outside [0, num_pages) sets LIN_ST_BAD_PAGE
 * and that page's tokens count as not seen.
 * Precision: scores, the softmax and the sums over values are fp32. bf16
 * caches multiply on tensor cores with exact bf16 operands and the weights in
 * two bf16 parts (three for fp32 outputs); fp32 caches multiply with every
 * operand in two tf32 parts. The sums of 16 tokens, and for fp32 caches of 32
 * channels of a score, are added with rounding; but bf16 outputs of more than 16
 * rows (n_q * num_q_heads / num_kv_heads) leave the value sums of up to 32,768
 * tokens to the tensor unit, which cuts off below the last place of fp32: less
 * than 2^-11 of the sum p |v|, where their own rounding is up to 2^-8. Visible NaN,
 * of any payload, gives NaN; visible infinities may give NaN, and values from
 * 2^120 on infinities, as weights relative to a lagging maximum reach 2^8.
 * Results do not depend on timing: the same call gives the same bits.
 * Any batch of lengths loads the SMs evenly: the lengths are read on the device,
 * the batch's tokens are cut into equal ranges, and items that cross a border
 * are joined by a second launch.
 * Workspace: lin_state_attn_workspace() bytes of device memory, 16-byte
 * aligned, not shared by calls that may overlap. The size never shrinks as
 * batch, n_q, num_q_heads / num_kv_heads or max_pages grow, and covers either
 * output type: one sized for the largest call serves the smaller ones. A few MB,
 * it depends on the GPU and not on the cache's size. Its contents
 * before the call do not matter. Longest request: 2^31 - 65536 tokens. */
typedef struct {
  int32_t layer, batch, n_q, num_q_heads;
  int32_t out_dtype;         /* lin_dtype_t */
  int32_t max_pages;         /* page table entries per request */
  float scale;               /* of q . k; 1/sqrt(head_dim) is usual */
  const void* q;             /* device */
  int64_t req_stride, token_stride; /* bytes, of q */
  void* out;                 /* device */
  const int32_t* page_table; /* device [batch], rows page_table_stride entries apart */
  int64_t page_table_stride;
  const int32_t* kv_len;     /* device [batch] */
  const int32_t* parent;     /* device [batch][n_q] or NULL */
  int32_t* status;
} lin_attn_args_t;

/* Bytes of workspace (0 for invalid arguments). Pointers in args are not read. */
LIN_API size_t lin_state_attn_workspace(const lin_kv_cache_t* cache, const lin_attn_args_t* args);
LIN_API int lin_state_attn_decode(const lin_kv_cache_t* cache, const lin_attn_args_t* args,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* ---- norms around a block ---------------------------------------------------
 * Per row of `channels` values, every part but x optional:
 *   t = x
 *   t = t * rsqrt(mean over its group of t^2 + eps) * w_post[c mod group]
 *   t = t * act(gate)                     (SiLU or sigmoid)
 *   h = residual + scale * scale_w[c] * t (residual 0 and scale_w 1 when NULL)
 *   y = h * rsqrt(mean over the row of h^2 + eps) * w_pre[c]
 * in fp32 throughout, rounded once where h_out and y are stored (y is made
 * from the unrounded h); the gate's sigmoid is 0 below -87.3. group divides channels: head_v for the output norm
 * of a linear-attention layer, channels for a norm after a block.
 * x is x_dtype; gate, the weights and y io_dtype; residual and h_out h_dtype.
 * Row strides in elements, at least `channels`; rows of any alignment do,
 * 16-byte aligned ones of whole 8-element vectors are faster. h_out may be
 * residual or x itself and y may be x or gate itself (same dtype and stride);
 * nothing else may overlap. channels <= 32768 (else LIN_EUNSUPPORTED). */
typedef enum { LIN_ACT_NONE = 0, LIN_ACT_SILU = 1, LIN_ACT_SIGMOID = 2 } lin_act_t;
typedef struct {
  int64_t rows;
  int32_t channels, group;   /* group: with w_post */
  int32_t x_dtype, io_dtype, h_dtype; /* lin_dtype_t */
  int32_t gate_act;          /* lin_act_t, with gate */
  float eps, scale;
  const void* x;             /* device */
  const void* gate;          /* device or NULL */
  const void* w_post;        /* device [group] or NULL */
  const void* residual;      /* device or NULL */
  const void* scale_w;       /* device [channels] or NULL */
  const void* w_pre;         /* device [channels] or NULL: no y */
  void* h_out;               /* device or NULL */
  void* y;                   /* device or NULL, with w_pre */
  int64_t x_stride, gate_stride, residual_stride, h_stride, y_stride; /* elements */
} lin_norm_args_t;

LIN_API int lin_state_block_norm(const lin_norm_args_t* args, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LIN_STEP_H_ */
