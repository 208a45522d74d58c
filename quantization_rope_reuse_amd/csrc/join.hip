// Attention over two parts of a cache made one.
//
// Rows and heads independent: 16 lanes take one vector (8 elements each), so
// a wave's loads and stores are whole 256-byte rows of 16-bit elements.  The
// weights e^(a - top) and e^(b - top) are at most 1, the larger of the two is
// 1, and the sum is divided out once, all in fp32.  Bytes bound it (16,381 tokens
// of 32 fp16 heads, 409 MB, in 71 us, 5.7 TB/s; 33 of 64 3 us, a launch's latency).
#include "hkv_device.h"
#include "pages_launch.h"

namespace hkv {
namespace {

constexpr int kVecLanes = 16;
constexpr float kLog2e = 1.44269504088896340736f;

struct JoinParams {
  HeadView a, b, out;
  const float* lse_a;
  const float* lse_b;
  float* lse;
  int64_t vecs;            // n_tokens * n_heads
  int32_t n_heads;
  double rcp_heads;
};

template <int DT>
__global__ __launch_bounds__(kThreads) void join_kernel(JoinParams p) {
  constexpr int ES = ElemSize<DT>::value;
  const int part = threadIdx.x & (kVecLanes - 1);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / kVecLanes);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / kVecLanes) + threadIdx.x / kVecLanes;
       i < p.vecs; i += step) {
    const float a = p.lse_a[i], b = p.lse_b[i];
    int64_t t = static_cast<int64_t>(static_cast<double>(i) * p.rcp_heads);
    int64_t h = i - t * p.n_heads;
    if (h < 0) {
      --t;
      h += p.n_heads;
    } else if (h >= p.n_heads) {
      ++t;
      h -= p.n_heads;
    }
    float x[8], y[8];
    load8<DT>(p.a.data + t * p.a.token + h * p.a.head + 8 * part * ES, x);
    load8<DT>(p.b.data + t * p.b.token + h * p.b.head + 8 * part * ES, y);
    const float top = fmaxf(a, b);
    // an infinite difference, or both parts empty: the terms below are 0 or 1
    float wa = a == top ? 1.0f : __builtin_amdgcn_exp2f((a - top) * kLog2e);
    float wb = b == top ? 1.0f : __builtin_amdgcn_exp2f((b - top) * kLog2e);
    if (a == -INFINITY) wa = 0.0f;
    if (b == -INFINITY) wb = 0.0f;
    const bool broken = a != a || b != b;
    const float sum = broken ? __builtin_nanf("") : wa + wb;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const float fa = wa * inv, fb = wb * inv;
    float z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float u = wa == 0.0f && !broken ? 0.0f : fa * x[j];
      const float v = wb == 0.0f && !broken ? 0.0f : fb * y[j];
      z[j] = u + v;
    }
    store8<DT>(p.out.data + t * p.out.token + h * p.out.head + 8 * part * ES, z);
    // sum is in [1, 2], or 0
    if (p.lse && part == 0) p.lse[i] = sum == 0.0f ? -INFINITY : top + logf(sum);
  }
}

}  // namespace

hipError_t launch_join(const HeadView& a, const float* lse_a, const HeadView& b, const float* lse_b,
                       int dtype, int32_t n_tokens, const HeadView& out, float* lse,
                       hipStream_t stream) {
  JoinParams p;
  p.a = a;
  p.b = b;
  p.out = out;
  p.lse_a = lse_a;
  p.lse_b = lse_b;
  p.lse = lse;
  p.n_heads = out.n_heads;
  p.vecs = static_cast<int64_t>(n_tokens) * out.n_heads;
  p.rcp_heads = 1.0 / out.n_heads;
  constexpr int64_t per_wg = kThreads / kVecLanes;
  // a launch holds less than 2^32 threads: vectors beyond 2^22 workgroups go round
  const int64_t need = (p.vecs + per_wg - 1) / per_wg;
  const dim3 grid(static_cast<unsigned>(need < (1 << 22) ? need : 1 << 22));
  switch (dtype) {
    case kF32: hipLaunchKernelGGL((join_kernel<kF32>), grid, dim3(kThreads), 0, stream, p); break;
    case kF16: hipLaunchKernelGGL((join_kernel<kF16>), grid, dim3(kThreads), 0, stream, p); break;
    default: hipLaunchKernelGGL((join_kernel<kBF16>), grid, dim3(kThreads), 0, stream, p);
  }
  return hipGetLastError();
}

}  // namespace hkv
