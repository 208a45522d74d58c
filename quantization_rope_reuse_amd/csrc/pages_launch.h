// Internal launch interface of the page serving calls (include/hkv_pages.h),
// between their checks (pages_api.hip) and the kernels.
#pragma once

#include "hkv_pages.h"
#include "serve_launch.h"

namespace hkv {

// rope NULL: no rotation (q then has no heads).
hipError_t launch_append_pages(const Geometry& g, const hkv_rope_axes* rope,
                               const int32_t* positions, int64_t axis_stride, const HeadView& q,
                               const HeadView& k, const HeadView& v, const HeadView& q_out,
                               int dtype, int32_t n_tokens, const int64_t* slots,
                               const PageView& dst, int dst_dtype, hipStream_t stream);

struct PageAttendCall {
  int dtype;
  Geometry g;
  PageView pages;
  hkv_requests req;
  hkv_scores scores;
  HeadView q, out;
  int32_t n_tokens;
  float* lse;              // may be NULL
  void* workspace;
};

int64_t attend_pages_workspace_bytes(const Geometry& g, const hkv_requests& req, int32_t n_tokens,
                                     int32_t n_q_heads, int dtype);
hipError_t launch_attend_pages(const PageAttendCall& c, hipStream_t stream);

hipError_t launch_join(const HeadView& a, const float* lse_a, const HeadView& b, const float* lse_b,
                       int dtype, int32_t n_tokens, const HeadView& out, float* lse,
                       hipStream_t stream);

}  // namespace hkv
