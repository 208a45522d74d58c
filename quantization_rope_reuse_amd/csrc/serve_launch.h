// Internal launch interface of the serving calls (include/hkv_serve.h),
// between their checks (serve_api.hip) and the kernels.
#pragma once

#include "hkv_launch.h"
#include "hkv_serve.h"

namespace hkv {

struct HeadView {          // byte addressing of rows of head vectors
  char* data;
  int64_t token, head;
  int32_t n_heads;
};

constexpr int32_t kMaxStepRequests = 4096;

hipError_t launch_plan(const hkv_step& s, hipStream_t stream);

hipError_t launch_rope(const hkv_rope_axes& rope, const int32_t* positions, int64_t axis_stride,
                       int32_t n_tokens, const HeadView& q, const HeadView& k,
                       const HeadView& q_out, const HeadView& k_out, int dtype, bool inverse,
                       hipStream_t stream);

hipError_t launch_append(int fmt, int dtype, const Geometry& g, const HeadView& k,
                         const HeadView& v, int32_t n_tokens, const int64_t* slots,
                         const RecordView& dst, hipStream_t stream);

struct AttendCall {
  int fmt;
  int dtype;
  Geometry g;
  RecordView rec;
  hkv_requests req;
  HeadView q, out;
  int32_t n_tokens;
  double sm_scale;
  bool causal;
  const int32_t* delta;    // NULL: stored positions stand
  double rope_base;
  int pairs;
  float* lse;              // may be NULL
  void* workspace;
};

int64_t attend_workspace_bytes(const Geometry& g, const hkv_requests& req, int32_t n_tokens,
                               int32_t n_q_heads, int dtype);
hipError_t launch_attend(const AttendCall& c, hipStream_t stream);

}  // namespace hkv
