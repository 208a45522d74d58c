/*
 * hkv_serve.h - serving from compressed records: the calls of one model step
 * that reads and extends a cache held as hkv records, without bringing it
 * back into pages.
 *
 *   plan    block tables, slots and positions of a step from its request
 *           lengths, with the blocks taken from and returned to a free list
 *           on the device (hkv_plan_step);
 *   rope    rotary positions with one or several axes for query and key
 *           heads (hkv_rope_heads);
 *   append  new tokens' keys and values quantized into their slots
 *           (hkv_append_tokens);
 *   attend  attention of queries over the records, stored keys optionally
 *           moved to new positions on the way (hkv_attend_records).
 *
 * The conventions of hkv.h hold for every call: device pointers owned by the
 * caller, asynchronous on `stream`, no allocation, no state between calls,
 * arguments checked on the host before anything is launched, the same status
 * codes, head_dim 128, no byte offset at or beyond 2^47.  Values that only
 * the device knows (lengths, table entries, slots) are never trusted: what
 * is out of range is skipped or clamped as each call says, and no access
 * leaves the given arrays.
 *
 * A pool of records is one layer's: the shape's n_layers must be 1 and its
 * n_blocks is the number of records in the pool.  A slot is a token's place
 * in the pool, block * block_tokens + token within the block.
 */
#ifndef HKV_SERVE_H
#define HKV_SERVE_H

#include "hkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of head vectors: element (token t, head h, dim j) at
 *   data + t*token_stride + h*head_stride + j
 * (strides in ELEMENTS, non-negative; the 128 elements contiguous).  data
 * and both strides times the element size: multiples of 16 bytes. */
typedef struct {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
  int32_t n_heads;       /* >= 0 */
} hkv_heads;

/* One step of a server's requests.  For request r, with
 *   len  = kv_len[r] clamped to [0, max_blocks * block_tokens],
 *   held = ceil(len / block_tokens):
 * new_tokens[r] < 0 ends it: its first `held` table entries are pushed onto
 *   the free list, kv_len_out[r] = 0.
 * new_tokens[r] = n >= 0 grows it by n tokens, which need
 *   need = ceil((len + n) / block_tokens) - held
 *   further blocks.
 * All pushes come first, in request order, then table order; pushes beyond
 * free_capacity are dropped.  Then blocks are popped off the top in the same
 * order into table entries held, held + 1, ...  A request is refused, and
 * takes nothing, if len + n exceeds max_blocks * block_tokens, or if it
 * needs blocks and the needs of all requests up to and including it (those
 * refused for their length not counted) exceed the list:
 *   refused[r] = 1, kv_len_out[r] = len.
 * Otherwise refused[r] = 0 and kv_len_out[r] = len + n.
 * Tokens are packed in request order, a refused request's included:
 * q_start[r] is the number of new tokens before request r (saturating at
 * 2^31 - 1), q_start[n_requests] their total.  For token i of them, the j-th
 * of request r (i < n_tokens; the rest of a longer step is not written):
 *   positions[i] = len + j,
 *   slots[i] = block_table[r][positions[i] / block_tokens] * block_tokens
 *              + positions[i] % block_tokens, or -1 if r is refused or that
 *              entry is negative;
 * entries from the total up to n_tokens get position 0 and slot -1.
 * kv_len, new_tokens and free_count are only read; the table and the list
 * change only as said (the list above free_count_out keeps its old entries),
 * so the same call on the same inputs gives the same result again.
 * n_requests above 4096, or max_blocks * block_tokens, n_requests *
 * max_blocks or n_tokens above 2^31 - 1: HKV_ERR_UNSUPPORTED. */
typedef struct {
  int32_t n_requests;          /* >= 0 */
  int32_t block_tokens;        /* >= 1 */
  int32_t max_blocks;          /* >= 0, entries per table row */
  int32_t n_tokens;            /* >= 0, entries of positions and slots */
  const int32_t* kv_len;       /* [n_requests] */
  const int32_t* new_tokens;   /* [n_requests] */
  int32_t* block_table;        /* [n_requests] rows of max_blocks */
  int64_t table_stride;        /* elements between rows, >= max_blocks */
  int32_t* free_blocks;        /* [free_capacity], a stack: top at the end */
  int32_t free_capacity;       /* >= 0 */
  const int32_t* free_count;   /* [1], clamped to [0, free_capacity] */
  int32_t* free_count_out;     /* [1], not free_count itself */
  int32_t* kv_len_out;         /* [n_requests], not kv_len itself */
  int32_t* q_start;            /* [n_requests + 1] */
  int32_t* positions;          /* [n_tokens] */
  int64_t* slots;              /* [n_tokens] */
  int32_t* refused;            /* [n_requests] */
} hkv_step;
int hkv_plan_step(const hkv_step* step, hipStream_t stream);

/* Rotary positions with several axes (time, height and width of an image or
 * video token; one axis for text).  Pair i of a head vector - elements
 * (2i, 2i+1) or (i, i+64), as hkv_rope_pairs - turns by
 *   phi_i = positions[axis[i]][t] / rope_base^(2 freq[i] / 128),
 *   (a, b) -> (a cos phi - b sin phi, a sin phi + b cos phi);
 * pairs with axis[i] = -1 and pairs whose angle is 0 pass through unchanged.
 * phi and its reduction modulo pi/2 are computed in double (for
 * |phi| < 2^31, off by about 2^-51 of phi), cos and sin of the reduced argument and the rotation in
 * fp32, and the result is rounded once to dtype. */
typedef struct {
  int32_t n_axes;        /* 1..8 */
  int32_t pairs;         /* hkv_rope_pairs */
  double rope_base;      /* finite, > 0 */
  int8_t axis[64];       /* -1 .. n_axes - 1 */
  uint8_t freq[64];      /* 0..127; pair i's own index i is the usual choice */
} hkv_rope_axes;

/* Rotates n_tokens rows of q and of k (either may have 0 heads) into q_out
 * and k_out, which may be q and k themselves (same data and strides) and
 * must not overlap them otherwise.  positions: int32, entry (axis a, token t)
 * at positions + a*axis_stride + t.  inverse != 0 turns by -phi: the
 * gradient of this call with respect to q and k, given that of its outputs
 * (a rotation's transpose), and the way to strip positions.  More than 2^24
 * heads in all, or n_tokens times them above 2^31 - 1: HKV_ERR_UNSUPPORTED. */
int hkv_rope_heads(const hkv_rope_axes* rope, const int32_t* positions, int64_t axis_stride,
                   int32_t n_tokens, const hkv_heads* q, const hkv_heads* k,
                   const hkv_heads* q_out, const hkv_heads* k_out, int32_t dtype,
                   int32_t inverse, hipStream_t stream);

/* Quantizes n_tokens rows of k and v (n_kv_heads heads each, one dtype) into
 * the pool: token t's vectors become the codes and scales of slot slots[t]
 * (int64, device), bit for bit what hkv_quant_fp8 / hkv_quant_int4 write for
 * the same vectors.  Slots outside [0, n_blocks * block_tokens) are skipped;
 * no two tokens may share a slot.  Other tokens of a block, their codes and
 * scales, are not touched.  n_tokens * n_kv_heads above 2^31 - 1:
 * HKV_ERR_UNSUPPORTED. */
int hkv_append_tokens(const hkv_shape* shape, int32_t fmt, const hkv_heads* k, const hkv_heads* v,
                      int32_t dtype, int32_t n_tokens, const int64_t* slots,
                      const hkv_records* dst, hipStream_t stream);

/* The requests of one attention call.  Request r's queries are the rows
 * q_start[r] .. q_start[r+1] - 1 of q (q_start NULL: row r alone, and
 * n_tokens must be n_requests); bounds outside [0, n_tokens] are clamped, a
 * range that is empty or backwards has no queries, and of a longer range
 * only the first max_queries rows are computed.  Its cached tokens are
 * 0 .. len - 1, len = kv_len[r] clamped to [0, max_blocks * block_tokens],
 * token m in record block_table[r][m / block_tokens] at m % block_tokens.
 * Tokens whose table entry is negative or >= n_blocks are left out, as if
 * masked.  Ranges of different requests must not overlap. */
typedef struct {
  int32_t n_requests;          /* >= 0 */
  int32_t max_blocks;          /* >= 0 */
  int32_t max_queries;         /* >= 1 */
  const int32_t* block_table;  /* [n_requests] rows of max_blocks */
  int64_t table_stride;        /* elements between rows, >= max_blocks */
  const int32_t* kv_len;       /* [n_requests] */
  const int32_t* q_start;      /* [n_requests + 1], or NULL */
} hkv_requests;

/* Stored keys moved to new positions while they are read, as
 * hkv_fetch_dequant_rope_shift moves them: every key of table entry (r, j)
 * turns by delta_m[r * table_stride + j] * theta_i.  (The call turns the
 * query by the opposite angle instead, which gives the same product.) */
typedef struct {
  const int32_t* delta_m;      /* rows as block_table's */
  double rope_base;            /* finite, > 0 */
  int32_t pairs;               /* hkv_rope_pairs */
} hkv_key_shift;

/* Attention over records.  Query head h reads key head h / (n_heads /
 * n_kv_heads).  For query row i, the j-th of n of its request, and head h:
 *   s_m = sm_scale * q_i,h . k_m   over the cached tokens m that it sees:
 *         all of them, or with causal != 0 those with m <= len - n + j;
 *   out = sum_m softmax(s)_m v_m,   lse = log sum_m exp(s_m);
 * a row that sees nothing gets out = 0 and lse = -infinity.  k_m and v_m are
 * code * scale, taken into the products exactly: codes enter the matrix
 * instructions as they are and scales multiply scores and weights in fp32.
 * Sums are fp32.  Queries enter scaled by a power of two: as two fp16 parts
 * (22 bits) where they are fp32 or turned by a shift, else as one, exact but
 * for elements far below their row's largest, which are off by at most 2^-38
 * of it (2^-24 in prompts, where rows of up to 2^14 in size share the power).
 * Weights enter as one fp16 part (11 bits) for bf16 results, as two for the
 * others.
 * What a token holds does not matter where its table entry is out of range or
 * where it stands past the end.  FP8 records must not hold NaN codes (0x7F,
 * 0xFF) elsewhere: rows that may not see the token yet, and another head's,
 * could become NaN with it.  hkv_quant_* and hkv_append_tokens write none: of a
 * vector with a NaN they make the scale NaN, which reaches what sees it alone.
 * q and out: dtype, n_tokens rows, the same number of heads, a multiple of
 * n_kv_heads; out must not overlap q.  lse: float [n_tokens][n_heads], or
 * NULL.  Rows of no request keep what out and lse held.
 * shift: NULL, or the keys' moves.  sm_scale: finite.
 * workspace: 16-byte aligned, hkv_attend_workspace_bytes() bytes (0: none
 * needed); its contents before and after do not matter, and calls that share
 * one must not overlap.  The result does not depend on scheduling: the same
 * call gives the same bits.  n_requests above 65535, n_kv_heads above 4096,
 * max_blocks * block_tokens or n_tokens * n_heads above 2^31 - 1:
 * HKV_ERR_UNSUPPORTED. */
int hkv_attend_records(const hkv_shape* shape, int32_t fmt, const hkv_records* records,
                       const hkv_requests* requests, const hkv_heads* q, int32_t dtype,
                       int32_t n_tokens, double sm_scale, int32_t causal,
                       const hkv_key_shift* shift, const hkv_heads* out, float* lse,
                       void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of hkv_attend_records for these sizes (pointers and
 * contents are not read); -1 on bad arguments. */
int64_t hkv_attend_workspace_bytes(const hkv_shape* shape, const hkv_requests* requests,
                                   int32_t n_tokens, int32_t n_q_heads, int32_t dtype);

#ifdef __cplusplus
}
#endif

#endif /* HKV_SERVE_H */
