// C ABI of the serving calls (include/hkv_serve.h): argument checks, all on
// the host before any HIP call, and dispatch to the launchers.
#include "hkv_serve.h"

#include <math.h>
#include <stdint.h>

#include "hkv_device.h"
#include "serve_launch.h"

namespace {

using hkv::Geometry;
using hkv::HeadView;
using hkv::RecordView;

bool aligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

int to_status(hipError_t e) { return e == hipSuccess ? HKV_OK : HKV_ERR_HIP; }

// Rows of head vectors; `data` may be NULL where nothing is addressed.
int check_heads(const hkv_heads* h, int32_t dtype, int32_t n_tokens, HeadView* v) {
  const int es = hkv::element_size(dtype);
  if (!h || es == 0 || h->n_heads < 0 || n_tokens < 0) return HKV_ERR_INVALID_ARG;
  for (int64_t s : {h->token_stride, h->head_stride}) {
    if (s < 0 || s > INT64_MAX / 8 || (s * es) % 16 != 0) return HKV_ERR_INVALID_ARG;
  }
  if (!aligned(h->data, 16)) return HKV_ERR_INVALID_ARG;
  if (!h->data && h->n_heads > 0 && n_tokens > 0) return HKV_ERR_INVALID_ARG;
  v->data = static_cast<char*>(h->data);
  v->token = h->token_stride * es;
  v->head = h->head_stride * es;
  v->n_heads = h->n_heads;
  if (!hkv::span_ok({{n_tokens, v->token}, {h->n_heads, v->head}}, int64_t{HKV_HEAD_DIM} * es))
    return HKV_ERR_INVALID_ARG;
  return HKV_OK;
}

// One layer's pool of records; an empty one addresses nothing, so its base
// may be NULL.
int check_pool(const hkv_shape* shape, int32_t fmt, const hkv_records* records, Geometry* g,
               RecordView* v) {
  int st;
  if ((st = hkv::shape_check(shape, g)) != HKV_OK) return st;
  if (g->n_layers != 1) return HKV_ERR_INVALID_ARG;
  if (records && g->n_blocks == 0) {
    *v = {nullptr, 0, 0};
    return hkv_record_bytes(fmt, g->block_tokens, g->n_heads, HKV_HEAD_DIM) < 0
               ? HKV_ERR_INVALID_ARG
               : HKV_OK;
  }
  return hkv::records_check(records, fmt, shape, v);
}

// Sizes of the requests of an attention call (pointers apart).
int check_requests(const hkv_requests* r, const Geometry& g, int32_t n_tokens, int32_t n_q_heads) {
  if (!r || r->n_requests < 0 || r->max_blocks < 0 || r->max_queries < 1 || n_tokens < 0 ||
      r->table_stride < r->max_blocks)
    return HKV_ERR_INVALID_ARG;
  if (n_q_heads < 1 || n_q_heads % g.n_heads != 0) return HKV_ERR_INVALID_ARG;
  if (r->n_requests > 65535) return HKV_ERR_UNSUPPORTED;                 // grid.y limit
  if (g.n_heads > 4096) return HKV_ERR_UNSUPPORTED;                      // grid.x limit
  if (static_cast<int64_t>(r->max_blocks) * g.block_tokens > INT32_MAX) return HKV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(n_tokens) * n_q_heads > INT32_MAX) return HKV_ERR_UNSUPPORTED;
  if (!hkv::span_ok({{r->n_requests, r->table_stride}}, r->max_blocks)) return HKV_ERR_INVALID_ARG;
  return HKV_OK;
}

}  // namespace

extern "C" {

int hkv_plan_step(const hkv_step* s, hipStream_t stream) {
  if (!s || s->n_requests < 0 || s->block_tokens < 1 || s->max_blocks < 0 || s->n_tokens < 0 ||
      s->free_capacity < 0 || s->table_stride < s->max_blocks)
    return HKV_ERR_INVALID_ARG;
  if (s->n_requests > hkv::kMaxStepRequests) return HKV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(s->max_blocks) * s->block_tokens > INT32_MAX ||
      static_cast<int64_t>(s->n_requests) * s->max_blocks > INT32_MAX)
    return HKV_ERR_UNSUPPORTED;
  if (!hkv::span_ok({{s->n_requests, s->table_stride}}, s->max_blocks)) return HKV_ERR_INVALID_ARG;
  if (!s->free_count || !s->free_count_out || s->free_count == s->free_count_out || !s->q_start)
    return HKV_ERR_INVALID_ARG;
  if (s->n_requests > 0 && (!s->kv_len || !s->new_tokens || !s->kv_len_out || !s->refused ||
                            s->kv_len == s->kv_len_out))
    return HKV_ERR_INVALID_ARG;
  if (s->n_requests > 0 && s->max_blocks > 0 && !s->block_table) return HKV_ERR_INVALID_ARG;
  if (s->free_capacity > 0 && !s->free_blocks) return HKV_ERR_INVALID_ARG;
  if (s->n_tokens > 0 && (!s->positions || !s->slots)) return HKV_ERR_INVALID_ARG;
  for (const void* q : {static_cast<const void*>(s->kv_len), static_cast<const void*>(s->new_tokens),
                        static_cast<const void*>(s->block_table),
                        static_cast<const void*>(s->free_blocks),
                        static_cast<const void*>(s->free_count),
                        static_cast<const void*>(s->free_count_out),
                        static_cast<const void*>(s->kv_len_out),
                        static_cast<const void*>(s->q_start),
                        static_cast<const void*>(s->positions),
                        static_cast<const void*>(s->refused)})
    if (!aligned(q, 4)) return HKV_ERR_INVALID_ARG;
  if (!aligned(s->slots, 8)) return HKV_ERR_INVALID_ARG;
  return to_status(hkv::launch_plan(*s, stream));
}

int hkv_rope_heads(const hkv_rope_axes* rope, const int32_t* positions, int64_t axis_stride,
                   int32_t n_tokens, const hkv_heads* q, const hkv_heads* k,
                   const hkv_heads* q_out, const hkv_heads* k_out, int32_t dtype,
                   int32_t inverse, hipStream_t stream) {
  if (!rope || rope->n_axes < 1 || rope->n_axes > 8) return HKV_ERR_INVALID_ARG;
  if (rope->pairs != HKV_ROPE_INTERLEAVED && rope->pairs != HKV_ROPE_HALF_SPLIT)
    return HKV_ERR_INVALID_ARG;
  if (!(rope->rope_base > 0.0) || !isfinite(rope->rope_base)) return HKV_ERR_INVALID_ARG;
  for (int i = 0; i < HKV_HEAD_DIM / 2; ++i)
    if (rope->axis[i] < -1 || rope->axis[i] >= rope->n_axes || rope->freq[i] > 127)
      return HKV_ERR_INVALID_ARG;
  HeadView v[4];
  const hkv_heads* heads[4] = {q, k, q_out, k_out};
  for (int i = 0; i < 4; ++i) {
    const int st = check_heads(heads[i], dtype, n_tokens, &v[i]);
    if (st != HKV_OK) return st;
  }
  if (q->n_heads != q_out->n_heads || k->n_heads != k_out->n_heads) return HKV_ERR_INVALID_ARG;
  if (axis_stride < 0 || !hkv::span_ok({{rope->n_axes, axis_stride}}, n_tokens) ||
      !aligned(positions, 4))
    return HKV_ERR_INVALID_ARG;
  const int64_t vecs = static_cast<int64_t>(q->n_heads) + k->n_heads;
  if (vecs > (1 << 24) || static_cast<int64_t>(n_tokens) * vecs > INT32_MAX)
    return HKV_ERR_UNSUPPORTED;
  if (n_tokens == 0 || vecs == 0) return HKV_OK;
  if (!positions) return HKV_ERR_INVALID_ARG;
  return to_status(hkv::launch_rope(*rope, positions, axis_stride, n_tokens, v[0], v[1], v[2], v[3],
                                    dtype, inverse != 0, stream));
}

int hkv_append_tokens(const hkv_shape* shape, int32_t fmt, const hkv_heads* k, const hkv_heads* v,
                      int32_t dtype, int32_t n_tokens, const int64_t* slots,
                      const hkv_records* dst, hipStream_t stream) {
  Geometry g;
  RecordView rv;
  HeadView kv, vv;
  int st;
  if ((st = check_pool(shape, fmt, dst, &g, &rv)) != HKV_OK) return st;
  if ((st = check_heads(k, dtype, n_tokens, &kv)) != HKV_OK) return st;
  if ((st = check_heads(v, dtype, n_tokens, &vv)) != HKV_OK) return st;
  if (k->n_heads != g.n_heads || v->n_heads != g.n_heads) return HKV_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n_tokens) * g.n_heads > INT32_MAX) return HKV_ERR_UNSUPPORTED;
  if (!aligned(slots, 8)) return HKV_ERR_INVALID_ARG;
  if (n_tokens == 0 || g.n_blocks == 0) return HKV_OK;
  if (!slots) return HKV_ERR_INVALID_ARG;
  return to_status(hkv::launch_append(fmt, dtype, g, kv, vv, n_tokens, slots, rv, stream));
}

int64_t hkv_attend_workspace_bytes(const hkv_shape* shape, const hkv_requests* requests,
                                   int32_t n_tokens, int32_t n_q_heads, int32_t dtype) {
  Geometry g;
  if (hkv::shape_check(shape, &g) != HKV_OK || g.n_layers != 1 || hkv::element_size(dtype) == 0 ||
      check_requests(requests, g, n_tokens, n_q_heads) != HKV_OK)
    return -1;
  return hkv::attend_workspace_bytes(g, *requests, n_tokens, n_q_heads, dtype);
}

int hkv_attend_records(const hkv_shape* shape, int32_t fmt, const hkv_records* records,
                       const hkv_requests* requests, const hkv_heads* q, int32_t dtype,
                       int32_t n_tokens, double sm_scale, int32_t causal,
                       const hkv_key_shift* shift, const hkv_heads* out, float* lse,
                       void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  hkv::AttendCall c;
  int st;
  if ((st = check_pool(shape, fmt, records, &c.g, &c.rec)) != HKV_OK) return st;
  if ((st = check_heads(q, dtype, n_tokens, &c.q)) != HKV_OK) return st;
  if ((st = check_heads(out, dtype, n_tokens, &c.out)) != HKV_OK) return st;
  if (q->n_heads != out->n_heads) return HKV_ERR_INVALID_ARG;
  if ((st = check_requests(requests, c.g, n_tokens, q->n_heads)) != HKV_OK) return st;
  if (!requests->q_start && requests->n_requests != n_tokens) return HKV_ERR_INVALID_ARG;
  if (!isfinite(static_cast<float>(sm_scale))) return HKV_ERR_INVALID_ARG;
  c.delta = nullptr;
  c.rope_base = 1.0;
  c.pairs = HKV_ROPE_HALF_SPLIT;
  if (shift) {
    if (!(shift->rope_base > 0.0) || !isfinite(shift->rope_base) || !aligned(shift->delta_m, 4) ||
        (shift->pairs != HKV_ROPE_INTERLEAVED && shift->pairs != HKV_ROPE_HALF_SPLIT))
      return HKV_ERR_INVALID_ARG;
    c.delta = shift->delta_m;
    c.rope_base = shift->rope_base;
    c.pairs = shift->pairs;
  }
  if (!aligned(requests->block_table, 4) || !aligned(requests->kv_len, 4) ||
      !aligned(requests->q_start, 4) || !aligned(lse, 4))
    return HKV_ERR_INVALID_ARG;
  if (requests->n_requests == 0 || n_tokens == 0) return HKV_OK;
  if (!requests->kv_len || (!requests->block_table && requests->max_blocks > 0) ||
      (shift && !shift->delta_m && requests->max_blocks > 0))
    return HKV_ERR_INVALID_ARG;
  const int64_t need =
      hkv::attend_workspace_bytes(c.g, *requests, n_tokens, q->n_heads, dtype);
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
    return HKV_ERR_INVALID_ARG;
  c.fmt = fmt;
  c.dtype = dtype;
  c.req = *requests;
  c.n_tokens = n_tokens;
  c.sm_scale = sm_scale;
  c.causal = causal != 0;
  c.lse = lse;
  c.workspace = workspace;
  return to_status(hkv::launch_attend(c, stream));
}

}  // extern "C"
