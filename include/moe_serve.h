/*
 * moe_serve.h — C ABI of the operators that stand around the routed layer of
 * moe_mxfp4.h in a serving step, exported by the same libmoe_mxfp4.so:
 *
 *   moe_kv_append        new keys and values into a paged cache, rotary
 *                        positions applied on the way (and to the queries)
 *   moe_prefix_attention attention of a batch whose sequences share a prefix,
 *                        over that cache
 *   moe_sample           one token per row of logits from given uniform
 *                        numbers, with temperature, top-k, top-p and min-p
 *
 * A step: project (the caller's product) -> moe_kv_append ->
 * moe_prefix_attention -> project -> moe_forward -> ... -> moe_sample.
 *
 * Conventions (where they differ from moe_mxfp4.h):
 *   - Pointers inside the host structs are DEVICE pointers; the structs are
 *     read during the call only.
 *   - `status` is a DEVICE int32 or NULL.  A problem that a kernel finds
 *     (MOE_ERR_DEVICE_CHECK: a page id, length or position out of range;
 *     MOE_ERR_TIMEOUT: a bounded wait that gave up) is stored there if it
 *     holds 0; the calls never clear it, so one read can cover many steps.
 *     What such a problem touches is skipped, never read or written out of
 *     range; the outputs it belongs to are unspecified.
 *   - Lengths, tables and sampling parameters are read on the device, so a
 *     captured graph follows their values; shapes, strides and prefix_len are
 *     taken at the call.
 */
#ifndef MOE_SERVE_H
#define MOE_SERVE_H

#include "moe_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A paged cache of bf16 keys and values.  Element (page, token, head, d) of
 * either is at page * page_stride + token * token_stride + head * head_stride
 * + d (elements; strides are multiples of 8, k and v 16-byte aligned, so the
 * token-major and the head-major order are both taken).  page_size: 16, 32,
 * 64 or 128 tokens; head_dim: 64 or 128; kv_heads <= 256. */
typedef struct {
  void* k;
  void* v;
  int32_t num_pages, page_size, kv_heads, head_dim;
  int64_t page_stride, token_stride, head_stride;
} moe_kv_cache;

/* A batch of sequences over one cache.  Every sequence sees the shared prefix
 * (prefix_len tokens in the pages of prefix_table), then its own part (kv_len[b]
 * tokens in the pages of row b of `table`).  Its q_len[b] new tokens are the
 * last ones of its own part: token i of them (0 <= i < q_len[b]) is own token
 * kv_len[b] - q_len[b] + i, at position prefix_len + that.
 *   batch        sequences, 1 .. 4096
 *   tokens       new tokens of all sequences together (the rows of q, k, v)
 *   max_q        an upper bound of q_len[b], >= 1; checked on the device
 *   table_stride entries between rows of `table`; table_pages: entries of a row
 *   q_start      [batch + 1] first row of each sequence, q_start[0] = 0,
 *                q_start[batch] = tokens; NULL: one token each (tokens == batch)
 *   prefix_len   0: no shared part (prefix_table may be NULL) */
typedef struct {
  int32_t batch, tokens, max_q, table_stride, table_pages, prefix_len;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* table;
  const int32_t* prefix_table;
} moe_kv_batch;

#define MOE_SERVE_MAX_BATCH 4096
#define MOE_SERVE_MAX_LEN (1 << 30) /* tokens of the prefix, and of an own part that attention reads */
#define MOE_SAMPLE_MAX_VOCAB 262144

/* Append: for every new token, k (rotated) and v go to the token's place in
 * the cache, and q (rotated) to q_out.
 *   x_dtype      of q, k and v (MOE_DT_F32 / MOE_DT_BF16); the arithmetic is
 *                fp32, rounded once to bf16
 *   q, q_out     [tokens][q_heads][head_dim]; both NULL: keys and values only.
 *                q_out is bf16 and may be q itself (bf16, the same stride);
 *                its rows must not overlap.
 *   *_stride     elements between tokens; heads lie head_dim apart.  Pointers
 *                are 16-byte aligned, strides a multiple of 16 bytes.
 *   rope         [rope_rows][rot_dim] fp32: row p holds the rot_dim / 2 cosines
 *                of position p, then the sines.  The first rot_dim values of a
 *                head are rotated: value i with i + rot_dim / 2, or, when
 *                interleaved, 2i with 2i + 1:
 *                  a' = a cos - b sin,  b' = b cos + a sin
 *                rot_dim: a multiple of 16 up to head_dim; 0 (rope NULL): none.
 * A token whose position is not below rope_rows (when rotating), whose place is
 * outside its table row, or whose page id is outside the cache is skipped and
 * reported (MOE_ERR_DEVICE_CHECK). */
int moe_kv_append(const moe_kv_cache* cache, const moe_kv_batch* batch, int x_dtype, const void* q, const void* k,
                  const void* v, int q_heads, int64_t q_stride, int64_t k_stride, int64_t v_stride, void* q_out,
                  int64_t q_out_stride, const float* rope, int rope_rows, int rot_dim, int interleaved,
                  int32_t* status, void* stream);

/* Bytes of device workspace moe_prefix_attention needs (0: bad arguments).  A
 * function of batch, tokens, max_q, q_heads, kv_heads, head_dim and of whether
 * prefix_len is zero; nothing in it is kept from one call to the next. */
size_t moe_attention_workspace_bytes(const moe_kv_cache* cache, const moe_kv_batch* batch, int q_heads);

/* Attention.  Row (n, h): query n's head h, key head h / (q_heads / kv_heads).
 * It sees the whole prefix and the own tokens up to its own position:
 *   out[n][h] = sum_j exp(scale q.k_j - lse) v_j,
 *   lse[n][h] = log sum_j exp(scale q.k_j)
 * in fp32 statistics; the softmax weights enter the second product in bf16.
 * A row that sees nothing (kv_len[b] - q_len[b] + i < 0 and no prefix) gives
 * zeros and lse = -inf.  Cache rows past a sequence's length are never used,
 * whatever they hold, and an infinity or NaN in a new token's key or value
 * reaches only the rows that see the token.
 *   q, out       bf16 [tokens][q_heads][head_dim], *_stride elements between
 *                tokens (multiples of 8; 16-byte aligned pointers; rows of out
 *                must not overlap)
 *   scale        > 0; scale log2(e) finite in fp32
 *   lse          [tokens][q_heads] fp32 (natural logarithm) or NULL
 *   ws           moe_attention_workspace_bytes, 256-byte aligned, uninitialised
 * The sums of a row are joined in a fixed order: results are the same from run
 * to run on one device. */
int moe_prefix_attention(const moe_kv_cache* cache, const moe_kv_batch* batch, const void* q, int q_heads,
                         int64_t q_stride, float scale, void* out, int64_t out_stride, float* lse, void* ws,
                         size_t ws_bytes, int32_t* status, void* stream);

/* Sampling, one token per row.  With T = temperature[r] (1 where the array is
 * NULL), z_i = logit_i * (1 / T) in fp32, m = max z, and integer weights
 *   W_i = rint(exp(z_i - m) * 2^31),
 * so that every sum below is exact and its order does not matter.  NaN counts
 * as -inf; if some z_i = +inf those have W = 2^31 and all others 0.
 * Tokens are ranked by z descending, then by index; the kept ones are those
 * with W_i > 0 that pass, in this order,
 *   top_k[r] > 0:  rank < top_k
 *   top_p[r] < 1:  the sum of W of better ranks < top_p * (sum of W so far kept)
 *                  (the best token always passes every filter)
 *   min_p[r] > 0:  exp(z_i - m) >= min(min_p, 1)  (fp32)
 * and the result is the first token in index order at which the running sum of
 * kept W exceeds floor(u[r] * S), S their total.  T = 0: the best token.  A row
 * with nothing but -inf or NaN, or whose T is negative or NaN, gives token -1,
 * kept 0, logprob -inf and zero probabilities.
 *   logits       [rows][vocab], `stride` elements between rows, f32 or bf16
 *                (aligned to the element); vocab <= MOE_SAMPLE_MAX_VOCAB
 *   u            [rows] in [0, 1) (others are clamped into it; NaN as 0)
 *   temperature, top_k, top_p, min_p   [rows] or NULL (off); device
 *   token        [rows] int32
 *   logprob      [rows] fp32 or NULL: log(W_token / S)
 *   kept         [rows] int32 or NULL: tokens that passed
 *   probs        [rows][vocab] fp32 contiguous or NULL: W_i / S of the kept, else 0 */
int moe_sample(int rows, int vocab, const void* logits, int dtype, int64_t stride, const float* u,
               const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
               int32_t* token, float* logprob, int32_t* kept, float* probs, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_SERVE_H */
