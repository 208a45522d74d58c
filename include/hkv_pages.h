/*
 * hkv_pages.h - serving from pages: the calls of one model step on a cache
 * held in pages (hkv_pages), fetched there from records or never compressed.
 *
 *   append  queries and keys rotated, keys and values written to their slots
 *           (hkv_append_pages);
 *   attend  attention over the pages: decodes, drafts, chunks of prompts and
 *           rows picked for recomputing, with capped scores, a bias by
 *           distance, and documents, prefixes and windows as masks
 *           (hkv_attend_pages);
 *   join    attention over two parts of a cache made one, such as records and
 *           pages (hkv_join_attention).
 *
 * The conventions of hkv.h and hkv_serve.h hold for every call.  Pages are
 * one layer's: the shape's n_layers must be 1 and its n_blocks the number of
 * pages, num_pages (layer_stride is not used).  A slot is page * block_tokens
 * + token within the page.
 */
#ifndef HKV_PAGES_H
#define HKV_PAGES_H

#include "hkv_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Writes n_tokens rows of k and v (n_kv_heads heads each) to slots[t] (int64,
 * device) of the pages, the keys turned as hkv_rope_heads turns them on the
 * way, and turns q into q_out: one call in the place of hkv_rope_heads and
 * two copies.  Keys and queries are rounded once, from the fp32 rotation to
 * dst_dtype and dtype; values are converted from dtype to dst_dtype.
 * rope NULL: keys are only converted, and q and q_out must have no heads;
 * else positions and axis_stride as in hkv_rope_heads.  q_out may be q itself
 * (same data and strides) and must not overlap the inputs otherwise; no page
 * overlaps them.  Slots outside [0, n_blocks * block_tokens) are skipped
 * (their queries are turned all the same); no two tokens may share a slot.
 * Other tokens of a page are not touched.  More than 2^24 heads in all, or
 * n_tokens times them above 2^31 - 1: HKV_ERR_UNSUPPORTED. */
int hkv_append_pages(const hkv_shape* shape, const hkv_rope_axes* rope, const int32_t* positions,
                     int64_t axis_stride, const hkv_heads* q, const hkv_heads* k,
                     const hkv_heads* v, const hkv_heads* q_out, int32_t dtype, int32_t n_tokens,
                     const int64_t* slots, const hkv_pages* dst, int32_t dst_dtype,
                     hipStream_t stream);

/* What a query row sees, and how it scores it.  Row i, the j-th of n of a
 * request of len cached tokens, stands at
 *   pos = positions[i], or len - n + j where positions is NULL,
 * and sees the cached token m, 0 <= m < len, where its table entry is in
 * [0, num_pages) and
 *   m < prefix_len[r], or
 *   m >= begin[i] and (causal = 0 or m <= pos) and (window = 0 or m > pos - window).
 * A row whose given position is negative sees nothing.  Its score is
 *   x = sm_scale * q . k_m;  cap > 0: x = cap * tanh(x / cap);
 *   s = x - slopes[head] * |pos - m|.
 * |sm_scale| or |sm_scale| / cap above 2^100, or a cap above 2^100 or below
 * 2^-100: HKV_ERR_UNSUPPORTED. */
typedef struct {
  double sm_scale;             /* finite */
  double cap;                  /* 0: not capped; else finite, > 0 */
  int32_t causal;
  int32_t window;              /* >= 0 */
  const int32_t* positions;    /* [n_tokens], or NULL */
  const int32_t* begin;        /* [n_tokens], or NULL: 0 (first token of the row's document) */
  const int32_t* prefix_len;   /* [n_requests], or NULL: 0 */
  const float* slopes;         /* [n_q_heads], or NULL: 0 */
} hkv_scores;

/* Attention over pages.  Query head h reads key head h / (n_heads /
 * n_kv_heads); requests as in hkv_attend_records, their table's entries pages.
 *   out = sum_m softmax(s)_m v_m,   lse = log sum_m exp(s_m)
 * over the tokens the row sees; a row that sees nothing, or whose scores are
 * all -infinity, gets out = 0 and lse = -infinity.  q, out and the pages share
 * one dtype.  Products are exact and their sums, the softmax and its sums
 * fp32.  What leaves fp32's range is infinite: a sum of products, a score or a
 * slope times log2(e); a row that sees a score of +infinity is NaN, and one of
 * -infinity adds nothing.  Weights of 16-bit types enter their product as two
 * parts of the type, 16 bits or more, where the call's requests have fewer than
 * 64 rows of a key head each on average or the call is small, and rounded to the
 * type (8 bits, 11 in fp16) where they have more: one kernel takes the whole
 * call.  So decodes beside a long prompt are better given a call of their own,
 * for their precision and their time.  What tokens that a row does not see hold, infinities and
 * NaN included, does not reach it (where rows meet values that are not finite,
 * the call takes several times as long).  out must not overlap q.  lse: float
 * [n_tokens][n_heads], or NULL.  Rows of no request keep what out and lse
 * held.  workspace: 16-byte aligned, hkv_attend_pages_workspace_bytes() bytes
 * (0: none needed); its contents before and after do not matter, and calls
 * that share one must not overlap.  The same call gives the same bits.  Limits
 * as hkv_attend_records'. */
int hkv_attend_pages(const hkv_shape* shape, const hkv_pages* pages, const hkv_requests* requests,
                     const hkv_heads* q, int32_t dtype, int32_t n_tokens, const hkv_scores* scores,
                     const hkv_heads* out, float* lse, void* workspace, int64_t workspace_bytes,
                     hipStream_t stream);

/* Workspace bytes of hkv_attend_pages for these sizes (pointers and contents
 * are not read); -1 on bad arguments. */
int64_t hkv_attend_pages_workspace_bytes(const hkv_shape* shape, const hkv_requests* requests,
                                         int32_t n_tokens, int32_t n_q_heads, int32_t dtype);

/* Two attentions of the same queries over different tokens (out and lse of
 * hkv_attend_records or hkv_attend_pages, causal = 0 for the part that every
 * row sees whole) made that over all of them:
 *   lse = log(exp(lse_a) + exp(lse_b)),
 *   out = exp(lse_a - lse) out_a + exp(lse_b - lse) out_b.
 * A part whose lse is -infinity adds nothing, whatever its out holds; where
 * both are, out = 0 and lse = -infinity.  out_a, out_b, out: dtype, n_tokens
 * rows of the same number of heads; out may be out_a or out_b themselves and
 * lse lse_a or lse_b (same data and strides) and must not overlap them
 * otherwise.  lse_a, lse_b, lse: float [n_tokens][n_heads]; lse may be NULL.
 * n_tokens * n_heads above 2^31 - 1: HKV_ERR_UNSUPPORTED. */
int hkv_join_attention(const hkv_heads* out_a, const float* lse_a, const hkv_heads* out_b,
                       const float* lse_b, int32_t dtype, int32_t n_tokens, const hkv_heads* out,
                       float* lse, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* HKV_PAGES_H */
