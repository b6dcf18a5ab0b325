/*
 * lin_prompt.h -- what a prompt, whole or in chunks, needs of a hybrid model's
 * full-attention layers, beside lin_state_prefill of its linear layers and under
 * the conventions of lin_state.h and lin_step.h (memory, streams, errors, status
 * bits): block tables, positions and slot maps built on the device from the
 * requests' lengths, rotary positions with the new keys and values going into the
 * paged cache, and causal attention of a batch's newest tokens over it.
 *
 * Tokens are packed as in lin_state_prefill: request r's new tokens are the rows
 * cu_seqlens[r] .. cu_seqlens[r+1]. Lengths, counts and tables are read on the
 * device, so a captured graph follows them; arrays of `tokens` rows may have more
 * rows than the batch has tokens.
 */
#ifndef LIN_PROMPT_H_
#define LIN_PROMPT_H_

#include "lin_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- device status bit (with those of lin_state.h and lin_step.h) --------- */
#define LIN_ST_NO_PAGES 1024 /* the list of free pages ends before a request's need */

/* ---- block tables, positions and slot maps -----------------------------------
 * Request r has length[r] cached tokens and gets n_new[r] more (n_new NULL: n each).
 * Its table holds pages for the cached ones; the pages that the new ones need,
 * ceil((length + new) / page_size) - ceil(length / page_size), are taken from
 * free_pages in request order and written behind them in page_table[r] (free_pages
 * NULL: the table holds them already). Written:
 *   cu_seqlens [batch+1] the running sum of the new tokens;
 *   kv_len [batch]       length + new: what attention over the cache takes;
 *   position, slot [tokens]  of every new token, packed: its position (length[r] + j,
 *                        or, with `parent` (device [batch][n], n <= 32, no n_new; the
 *                        trees of lin_decode_args_t), length[r] + the draft's depth)
 *                        and its row of the cache, page * page_size + row in the page
 *                        of token length[r] + j; both -1 in rows past the last token;
 *   taken [1]            pages taken: free_pages[0 .. taken) are in use now.
 * cu_seqlens, kv_len, position, slot and taken may be NULL. Table entries behind a
 * request's pages are left as they are.
 * length[r] < 0 marks padding: no tokens, kv_len -1. Left out (kv_len -1, positions
 * and slots -1, no pages; its rows still count in cu_seqlens) is a request
 *   with a negative n_new (counted as 0), with more tokens than max_pages pages hold,
 *   or past row `tokens`: LIN_ST_BAD_SEQLEN;
 *   whose tree breaks its rules: LIN_ST_BAD_TREE;
 *   for which free pages are short: LIN_ST_NO_PAGES (those after it that need pages
 *   are short of them too).
 * A page id outside [0, num_pages), in the list or in the table, sets
 * LIN_ST_BAD_PAGE, and its tokens' slots are -1. kv_len must not be `length`, nor
 * overlap any other input: they are read while it is written. */
typedef struct {
  int32_t batch, n, tokens;
  int32_t page_size, num_pages;
  int32_t max_pages;         /* page table entries per request */
  int32_t num_free;          /* entries of free_pages */
  const int32_t* length;     /* device [batch] */
  const int32_t* n_new;      /* device [batch] or NULL */
  const int32_t* parent;     /* device [batch][n] or NULL */
  int32_t* page_table;       /* device [batch], rows page_table_stride entries apart */
  int64_t page_table_stride;
  const int32_t* free_pages; /* device [num_free] or NULL */
  int32_t* taken;            /* device [1] or NULL */
  int32_t* cu_seqlens;       /* device [batch+1] or NULL */
  int32_t* kv_len;           /* device [batch] or NULL */
  int32_t* position;         /* device [tokens] or NULL */
  int64_t* slot;             /* device [tokens] or NULL */
  int32_t* status;
} lin_kv_plan_args_t;

LIN_API int lin_state_kv_plan(const lin_kv_plan_args_t* args, void* stream);

/* ---- rotary positions, and the append of the turned keys ------------------------
 * For every token t with position[t] >= 0, every head of q and k and every pair
 * i < rot_dim / 2 of its channels, (i, i + rot_dim / 2) in the half layout, (2 i,
 * 2 i + 1) in the interleaved one, with a = position[t] * inv_freq[i]:
 *   (x, y) -> scale (x cos a - y sin a, y cos a + x sin a);
 * channels from rot_dim on stay as they are. position[t] < 0 marks padding: nothing
 * of that token is written.
 * The angle is reduced in 64-bit fixed point, so that cosine and sine are off by less
 * than 2^-22 at any position (inv_freq finite, below 16 in magnitude); products are
 * fp32, rounded once.
 * q, k, v [tokens][heads][head_dim] in `dtype`, a token's heads contiguous, token
 * strides in bytes. Each of these is optional:
 *   q_out       the turned queries (q itself may be given);
 *   k_out       the turned keys (k itself may be given);
 *   cache, slot the turned keys, and v as it is, go to row slot[t] of the cache's
 *               `layer` (slot < 0: not written; past the last page LIN_ST_BAD_PAGE).
 *               No two tokens may have the same slot. The cache has num_k_heads heads
 *               of head_dim in dtype.
 * head_dim is a multiple of 8 up to 256, rot_dim even and at most head_dim. Addresses
 * and strides are multiples of 16 bytes. Apart from the exact q_out == q and
 * k_out == k (with the same stride) nothing written may overlap what is read. */
typedef struct {
  int32_t layer, tokens, num_q_heads, num_k_heads, head_dim, rot_dim;
  int32_t interleaved;       /* 0: half layout */
  int32_t dtype;             /* lin_dtype_t */
  float scale;
  const void* q;             /* device, with q_out */
  const void* k;             /* device, with k_out or a cache */
  const void* v;             /* device, with a cache */
  void* q_out;               /* device or NULL */
  void* k_out;               /* device or NULL */
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride; /* bytes */
  const int32_t* position;   /* device [tokens] */
  const float* inv_freq;     /* device [rot_dim / 2] */
  const int64_t* slot;       /* device [tokens], with a cache */
  int32_t* status;
} lin_rope_args_t;

/* cache: NULL where nothing is appended. */
LIN_API int lin_state_rope(const lin_kv_cache_t* cache, const lin_rope_args_t* args, void* stream);

/* ---- attention of a chunk of new tokens -------------------------------------------
 * Causal attention of each request's new tokens over its cached tokens, the new ones
 * included: append them first. Request r's n = cu_seqlens[r+1] - cu_seqlens[r] queries
 * are its newest tokens: query i lies at position kv_len[r] - n + i and sees every
 * token up to its own. Query head h reads key-value head
 * h / (num_q_heads / num_kv_heads).
 * out[row][h] = sum_t softmax_t(scale q . k_t) v_t; a query that sees nothing
 * (kv_len < n) gives zeros. Keys and values that a query does not see have no part in
 * its output, whatever they hold (NaN too).
 * q [tokens][num_q_heads][head_dim] has the cache's dtype, token stride in bytes (a
 * multiple of 16); out is contiguous, in out_dtype. Rows that belong to no request
 * are left as they are, and so is a request with kv_len[r] < 0 (padding) or one with
 * a kv_len past max_pages * page_size or rows outside [0, tokens], in no rising order
 * (LIN_ST_BAD_SEQLEN). A page id outside [0, num_pages) sets LIN_ST_BAD_PAGE and that
 * page's tokens count as not seen.
 * Precision: scores, the softmax and the sums over values are fp32. bf16 caches with
 * bf16 outputs multiply on tensor cores with the weights rounded to bf16 (2^-8 at most,
 * 2^-9 rms; their sum is that of the unrounded ones), and the tensor unit's own value
 * sums, which cut off below the last place of fp32, end after 32,768 tokens at most: less
 * than 2^-11 of the sum p |v| at any length. fp32 outputs take the weights in three bf16
 * parts, fp32 caches every operand in two tf32 parts, and add every 16 tokens with
 * rounding. Visible NaN give NaN; visible infinities may, and values from 2^120 on
 * infinities. Results do not depend on timing: the same call gives the same bits. Nor does
 * a row depend on what other rows see.
 * Lengths are read on the device. The batch's work is cut into equal ranges for the SMs,
 * and blocks of queries that cross a border are joined by a second launch. Where `tokens`
 * allows many blocks for each SM (bf16 outputs), a launch in front looks whether the lengths
 * do: if so, whole blocks are taken one by one from a counter in the workspace. Which way,
 * and the rows of a block, go by batch, tokens, num_q_heads, max_pages and the lengths: the
 * same tokens in a call with other room may differ in their last bits.
 * bf16 outputs: pages of a multiple of 8 tokens load faster (by TMA) than others, and so do
 * queries whose heads per kv head divide 128 (with 7 of them a prompt takes 1.2 times as
 * long for its work as with 8). fp32 outputs of a bf16 cache take 2 to 6 times as long.
 * out must not overlap anything that is read.
 * Workspace: lin_state_attn_chunk_workspace() bytes of device memory, 16-byte aligned,
 * not shared by calls that may overlap. The size never shrinks as batch, tokens,
 * num_q_heads or max_pages grow and covers either output type, some 40 MB at most (152 SMs). Its
 * contents before the call do not matter. Longest request: 2^31 - 65536 tokens. */
typedef struct {
  int32_t layer, batch, tokens, num_q_heads;
  int32_t out_dtype;         /* lin_dtype_t */
  int32_t max_pages;         /* page table entries per request */
  float scale;               /* of q . k; 1/sqrt(head_dim) is usual */
  const void* q;             /* device */
  int64_t token_stride;      /* bytes, of q */
  void* out;                 /* device */
  const int32_t* page_table; /* device [batch], rows page_table_stride entries apart */
  int64_t page_table_stride;
  const int32_t* cu_seqlens; /* device [batch+1] */
  const int32_t* kv_len;     /* device [batch] */
  int32_t* status;
} lin_attn_chunk_args_t;

/* Bytes of workspace (0 for invalid arguments). Pointers in args are not read. */
LIN_API size_t lin_state_attn_chunk_workspace(const lin_kv_cache_t* cache, const lin_attn_chunk_args_t* args);
LIN_API int lin_state_attn_chunk(const lin_kv_cache_t* cache, const lin_attn_chunk_args_t* args,
                                 void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LIN_PROMPT_H_ */
