// Rotary positions with several axes for query and key heads.
//
// Pair i of every head vector of token t turns by the position of token t on
// the pair's axis times theta_i.  The angles depend on the token and the
// pair alone, so a wave takes vectors of one token: lane i computes pair i's
// cosine and sine once, each lane gathers the 8 it needs across the wave
// (lane layout of hkv_device.h: both pair conventions keep a pair inside one
// lane), and 8 vectors are loaded, turned in fp32 and stored.  The inverse,
// which is also the gradient, changes the sine's sign.
//
// Bytes bound it: every element is read once and written once (40 heads of
// 24,571 tokens in fp16: 84 us, 6.0 TB/s of the 6.2 that a large elementwise
// pass reaches; torch's copy 5.1).
// Stores pass the caches by (non-temporal), 4 % faster on large calls than
// plain ones; one vector a lane group is as fast as two, three or five.
#include "rope_device.h"
#include "serve_launch.h"

namespace hkv {
namespace {

struct RopeParams {
  const char* q;
  const char* k;
  char* q_out;
  char* k_out;
  int64_t q_token, q_head, k_token, k_head;
  int64_t qo_token, qo_head, ko_token, ko_head;
  int32_t q_heads, vecs;        // vectors of a token: q's, then k's
  int32_t chunks;               // waves of a token, 8 vectors each
  int64_t waves;
  const int32_t* positions;
  int64_t axis_stride;
  float sign;
  int8_t axis[kHeadDim / 2];
  double theta[kHeadDim / 2];   // quarter turns per position; 0 where axis is -1
};

template <int DT, int PAIRS>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeParams p) {
  constexpr int ES = ElemSize<DT>::value;
  const int lane = threadIdx.x & (kWave - 1);
  const int sub = lane & (kLanesPerVec - 1);
  const int vsub = lane / kLanesPerVec;
  const int axis = p.axis[lane];
  const double theta = p.theta[lane];
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / kWave);
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / kWave) + threadIdx.x / kWave;
       w < p.waves; w += step) {
    const int64_t t = w / p.chunks;
    const int v = static_cast<int>(w - t * p.chunks) * kVecsPerWave + vsub;
    const bool is_q = v < p.q_heads;
    const int h = is_q ? v : v - p.q_heads;
    const char* src = is_q ? p.q + t * p.q_token + h * p.q_head : p.k + t * p.k_token + h * p.k_head;
    char* dst = is_q ? p.q_out + t * p.qo_token + h * p.qo_head
                     : p.k_out + t * p.ko_token + h * p.ko_head;
    float a[8] = {}, b[8] = {};
    if (v < p.vecs) {
      load8<DT>(src + 8 * sub * ES, a);
      load8<DT>(src + (64 + 8 * sub) * ES, b);
    }
    const int pos = axis < 0 ? 0 : p.positions[axis * p.axis_stride + t];
    float c, s;
    cos_sin(pos, theta, &c, &s);
    s *= p.sign;
    float cs[8], sn[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cs[j] = __shfl(c, lane_pair(PAIRS, sub, j));
      sn[j] = __shfl(s, lane_pair(PAIRS, sub, j));
    }
    turn_runs<PAIRS>(a, b, cs, sn);
    if (v < p.vecs) {
      store8<DT, true>(dst + 8 * sub * ES, a);
      store8<DT, true>(dst + (64 + 8 * sub) * ES, b);
    }
  }
}

template <int DT>
hipError_t launch_dt(int pairs, const RopeParams& p, unsigned wgs, hipStream_t stream) {
  if (pairs == kInterleaved)
    hipLaunchKernelGGL((rope_kernel<DT, kInterleaved>), dim3(wgs), dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((rope_kernel<DT, kHalfSplit>), dim3(wgs), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const hkv_rope_axes& rope, const int32_t* positions, int64_t axis_stride,
                       int32_t n_tokens, const HeadView& q, const HeadView& k,
                       const HeadView& q_out, const HeadView& k_out, int dtype, bool inverse,
                       hipStream_t stream) {
  RopeParams p;
  p.q = q.data;
  p.k = k.data;
  p.q_out = q_out.data;
  p.k_out = k_out.data;
  p.q_token = q.token;
  p.q_head = q.head;
  p.k_token = k.token;
  p.k_head = k.head;
  p.qo_token = q_out.token;
  p.qo_head = q_out.head;
  p.ko_token = k_out.token;
  p.ko_head = k_out.head;
  p.q_heads = q.n_heads;
  p.vecs = q.n_heads + k.n_heads;
  p.positions = positions;
  p.axis_stride = axis_stride;
  p.sign = inverse ? -1.0f : 1.0f;
  for (int i = 0; i < kHeadDim / 2; ++i) {
    p.axis[i] = rope.axis[i];
    p.theta[i] = rope.axis[i] < 0 ? 0.0 : quarter_turns(rope.rope_base, rope.freq[i]);
  }
  p.chunks = (p.vecs + kVecsPerWave - 1) / kVecsPerWave;
  p.waves = static_cast<int64_t>(n_tokens) * p.chunks;
  // a launch holds less than 2^32 threads: waves beyond 2^22 workgroups go round
  const int64_t need = (p.waves + kThreads / kWave - 1) / (kThreads / kWave);
  const unsigned wgs = static_cast<unsigned>(need < (1 << 22) ? need : 1 << 22);
  switch (dtype) {
    case kF32: return launch_dt<kF32>(rope.pairs, p, wgs, stream);
    case kF16: return launch_dt<kF16>(rope.pairs, p, wgs, stream);
    default: return launch_dt<kBF16>(rope.pairs, p, wgs, stream);
  }
}

}  // namespace hkv
