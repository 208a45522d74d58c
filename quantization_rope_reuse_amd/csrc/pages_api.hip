// C ABI of the page serving calls (include/hkv_pages.h): argument checks, all
// on the host before any HIP call, and dispatch to the launchers.
#include "hkv_pages.h"

#include <math.h>
#include <stdint.h>

#include "pages_launch.h"

namespace {

using hkv::Geometry;
using hkv::HeadView;
using hkv::PageView;

bool aligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

int to_status(hipError_t e) { return e == hipSuccess ? HKV_OK : HKV_ERR_HIP; }

// One layer's pages; a pool of none addresses nothing, so its arrays may be NULL.
int check_pool(const hkv_shape* shape, const hkv_pages* pages, int32_t dtype, Geometry* g, PageView* v) {
  int st;
  if ((st = hkv::shape_check(shape, g)) != HKV_OK) return st;
  if (g->n_layers != 1 || !pages || pages->num_pages != g->n_blocks || hkv::element_size(dtype) == 0)
    return HKV_ERR_INVALID_ARG;
  if (g->n_blocks == 0) {
    *v = {};
    return HKV_OK;
  }
  return hkv::pages_check(pages, dtype, shape, v);
}

}  // namespace

extern "C" {

int hkv_append_pages(const hkv_shape* shape, const hkv_rope_axes* rope, const int32_t* positions,
                     int64_t axis_stride, const hkv_heads* q, const hkv_heads* k,
                     const hkv_heads* v, const hkv_heads* q_out, int32_t dtype, int32_t n_tokens,
                     const int64_t* slots, const hkv_pages* dst, int32_t dst_dtype,
                     hipStream_t stream) {
  Geometry g;
  PageView pv;
  HeadView qv, kv, vv, ov;
  int st;
  if ((st = check_pool(shape, dst, dst_dtype, &g, &pv)) != HKV_OK) return st;
  if ((st = hkv::heads_check(q, dtype, n_tokens, &qv)) != HKV_OK) return st;
  if ((st = hkv::heads_check(q_out, dtype, n_tokens, &ov)) != HKV_OK) return st;
  if ((st = hkv::heads_check(k, dtype, n_tokens, &kv)) != HKV_OK) return st;
  if ((st = hkv::heads_check(v, dtype, n_tokens, &vv)) != HKV_OK) return st;
  if (k->n_heads != g.n_heads || v->n_heads != g.n_heads || q->n_heads != q_out->n_heads)
    return HKV_ERR_INVALID_ARG;
  if (rope) {
    if ((st = hkv::rope_check(rope, positions, axis_stride, n_tokens)) != HKV_OK) return st;
  } else if (q->n_heads != 0) {
    return HKV_ERR_INVALID_ARG;
  }
  if (!aligned(slots, 8)) return HKV_ERR_INVALID_ARG;
  const int64_t vecs = static_cast<int64_t>(q->n_heads) + 2 * static_cast<int64_t>(g.n_heads);
  if (vecs > (1 << 24) || static_cast<int64_t>(n_tokens) * vecs > INT32_MAX) return HKV_ERR_UNSUPPORTED;
  if (n_tokens == 0) return HKV_OK;
  if ((rope && !positions) || !slots) return HKV_ERR_INVALID_ARG;
  return to_status(hkv::launch_append_pages(g, rope, positions, axis_stride, qv, kv, vv, ov, dtype,
                                            n_tokens, slots, pv, dst_dtype, stream));
}

int64_t hkv_attend_pages_workspace_bytes(const hkv_shape* shape, const hkv_requests* requests,
                                         int32_t n_tokens, int32_t n_q_heads, int32_t dtype) {
  Geometry g;
  if (hkv::shape_check(shape, &g) != HKV_OK || g.n_layers != 1 || hkv::element_size(dtype) == 0 ||
      hkv::requests_check(requests, g, n_tokens, n_q_heads) != HKV_OK)
    return -1;
  return hkv::attend_pages_workspace_bytes(g, *requests, n_tokens, n_q_heads, dtype);
}

int hkv_attend_pages(const hkv_shape* shape, const hkv_pages* pages, const hkv_requests* requests,
                     const hkv_heads* q, int32_t dtype, int32_t n_tokens, const hkv_scores* scores,
                     const hkv_heads* out, float* lse, void* workspace, int64_t workspace_bytes,
                     hipStream_t stream) {
  hkv::PageAttendCall c;
  int st;
  if ((st = check_pool(shape, pages, dtype, &c.g, &c.pages)) != HKV_OK) return st;
  if ((st = hkv::heads_check(q, dtype, n_tokens, &c.q)) != HKV_OK) return st;
  if ((st = hkv::heads_check(out, dtype, n_tokens, &c.out)) != HKV_OK) return st;
  if (q->n_heads != out->n_heads) return HKV_ERR_INVALID_ARG;
  if ((st = hkv::requests_check(requests, c.g, n_tokens, q->n_heads)) != HKV_OK) return st;
  if (!requests->q_start && requests->n_requests != n_tokens) return HKV_ERR_INVALID_ARG;
  if (!scores || !isfinite(scores->sm_scale) || scores->window < 0 || !(scores->cap >= 0.0) || !isfinite(scores->cap))
    return HKV_ERR_INVALID_ARG;
  // what the kernels keep of scale and cap fits fp32
  if (fabs(scores->sm_scale) > 0x1p100 ||
      (scores->cap > 0.0 && (scores->cap > 0x1p100 || scores->cap < 0x1p-100 ||
                             fabs(scores->sm_scale) / scores->cap > 0x1p100)))
    return HKV_ERR_UNSUPPORTED;
  for (const void* x : {static_cast<const void*>(requests->block_table), static_cast<const void*>(requests->kv_len),
                        static_cast<const void*>(requests->q_start), static_cast<const void*>(scores->positions),
                        static_cast<const void*>(scores->begin), static_cast<const void*>(scores->prefix_len),
                        static_cast<const void*>(scores->slopes), static_cast<const void*>(lse)})
    if (!aligned(x, 4)) return HKV_ERR_INVALID_ARG;
  if (requests->n_requests == 0 || n_tokens == 0) return HKV_OK;
  if (!requests->kv_len || (!requests->block_table && requests->max_blocks > 0)) return HKV_ERR_INVALID_ARG;
  const int64_t need = hkv::attend_pages_workspace_bytes(c.g, *requests, n_tokens, q->n_heads, dtype);
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return HKV_ERR_INVALID_ARG;
  c.dtype = dtype;
  c.req = *requests;
  c.scores = *scores;
  c.n_tokens = n_tokens;
  c.lse = lse;
  c.workspace = workspace;
  return to_status(hkv::launch_attend_pages(c, stream));
}

int hkv_join_attention(const hkv_heads* out_a, const float* lse_a, const hkv_heads* out_b,
                       const float* lse_b, int32_t dtype, int32_t n_tokens, const hkv_heads* out,
                       float* lse, hipStream_t stream) {
  HeadView a, b, o;
  int st;
  if ((st = hkv::heads_check(out_a, dtype, n_tokens, &a)) != HKV_OK) return st;
  if ((st = hkv::heads_check(out_b, dtype, n_tokens, &b)) != HKV_OK) return st;
  if ((st = hkv::heads_check(out, dtype, n_tokens, &o)) != HKV_OK) return st;
  if (a.n_heads != o.n_heads || b.n_heads != o.n_heads) return HKV_ERR_INVALID_ARG;
  if (!aligned(lse_a, 4) || !aligned(lse_b, 4) || !aligned(lse, 4)) return HKV_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n_tokens) * o.n_heads > INT32_MAX) return HKV_ERR_UNSUPPORTED;
  if (n_tokens == 0 || o.n_heads == 0) return HKV_OK;
  if (!lse_a || !lse_b) return HKV_ERR_INVALID_ARG;
  return to_status(hkv::launch_join(a, lse_a, b, lse_b, dtype, n_tokens, o, lse, stream));
}

}  // extern "C"
