// Append to pages: queries and keys turned by their positions, keys and
// values written to their slots, in one launch.
//
// The rotation of rope.hip, with the vectors of a token three runs: its
// queries, keys and values.  A wave takes 8 vectors of one token, so a token's
// slot and angles are read and computed once per wave; value vectors turn by
// nothing.  Bytes bound it: every element is read once and written once (a prompt
// with images of 403 MB in 70 us, 5.7 TB/s; a decode step of 48 tokens 3.8 us, a
// launch's latency).
#include "pages_launch.h"
#include "rope_device.h"

namespace hkv {
namespace {

struct AppendPagesParams {
  HeadView q, k, v, q_out;
  char* page_k;
  char* page_v;
  int64_t page, token, head;
  const int64_t* slots;
  int64_t n_slots;
  double rcp_block;             // 1 / block_tokens
  int32_t block_tokens;
  int32_t q_heads, kv_heads, vecs;
  int32_t chunks;               // waves of a token, 8 vectors each
  int64_t waves;
  const int32_t* positions;
  int64_t axis_stride;
  int8_t axis[kHeadDim / 2];
  double theta[kHeadDim / 2];   // quarter turns per position; 0 where axis is -1
};

template <int SDT, int PDT, int PAIRS>
__global__ __launch_bounds__(kThreads) void append_pages_kernel(AppendPagesParams p) {
  constexpr int ES = ElemSize<SDT>::value, EP = ElemSize<PDT>::value;
  const int lane = threadIdx.x & (kWave - 1);
  const int sub = lane & (kLanesPerVec - 1);
  const int vsub = lane / kLanesPerVec;
  const int axis = p.axis[lane];
  const double theta = p.theta[lane];
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / kWave);
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / kWave) + threadIdx.x / kWave;
       w < p.waves; w += step) {
    const int64_t t = w / p.chunks;
    const int first = static_cast<int>(w - t * p.chunks) * kVecsPerWave;
    const int i = first + vsub;
    const bool is_q = i < p.q_heads;
    const bool is_k = !is_q && i < p.q_heads + p.kv_heads;
    const int h = is_q ? i : is_k ? i - p.q_heads : i - p.q_heads - p.kv_heads;
    const char* src = is_q   ? p.q.data + t * p.q.token + h * p.q.head
                      : is_k ? p.k.data + t * p.k.token + h * p.k.head
                             : p.v.data + t * p.v.token + h * p.v.head;
    float a[8] = {}, b[8] = {};
    if (i < p.vecs) {
      load8<SDT>(src + 8 * sub * ES, a);
      load8<SDT>(src + (64 + 8 * sub) * ES, b);
    }
    const int64_t slot = p.slots[t];
    if (first < p.q_heads + p.kv_heads) {          // some vector of the wave turns
      const int pos = axis < 0 ? 0 : p.positions[axis * p.axis_stride + t];
      float c, s;
      cos_sin(pos, theta, &c, &s);
      float cs[8], sn[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        cs[j] = __shfl(c, lane_pair(PAIRS, sub, j));
        sn[j] = __shfl(s, lane_pair(PAIRS, sub, j));
      }
      if (is_q || is_k) turn_runs<PAIRS>(a, b, cs, sn);
    }
    if (i >= p.vecs) continue;
    if (is_q) {
      char* dst = p.q_out.data + t * p.q_out.token + h * p.q_out.head;
      store8<SDT, true>(dst + 8 * sub * ES, a);
      store8<SDT, true>(dst + (64 + 8 * sub) * ES, b);
    } else if (slot >= 0 && slot < p.n_slots) {
      // the product is off by less than one from the quotient
      int64_t page = static_cast<int64_t>(static_cast<double>(slot) * p.rcp_block);
      int64_t at = slot - page * p.block_tokens;
      if (at < 0) {
        --page;
        at += p.block_tokens;
      } else if (at >= p.block_tokens) {
        ++page;
        at -= p.block_tokens;
      }
      char* dst = (is_k ? p.page_k : p.page_v) + page * p.page + at * p.token + h * p.head;
      store8<PDT, true>(dst + 8 * sub * EP, a);
      store8<PDT, true>(dst + (64 + 8 * sub) * EP, b);
    }
  }
}

template <int SDT, int PDT>
hipError_t launch_types(int pairs, const AppendPagesParams& p, dim3 grid, hipStream_t stream) {
  if (pairs == kInterleaved)
    hipLaunchKernelGGL((append_pages_kernel<SDT, PDT, kInterleaved>), grid, dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((append_pages_kernel<SDT, PDT, kHalfSplit>), grid, dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

template <int SDT>
hipError_t launch_source(int dst_dtype, int pairs, const AppendPagesParams& p, dim3 grid,
                         hipStream_t stream) {
  switch (dst_dtype) {
    case kF32: return launch_types<SDT, kF32>(pairs, p, grid, stream);
    case kF16: return launch_types<SDT, kF16>(pairs, p, grid, stream);
    default: return launch_types<SDT, kBF16>(pairs, p, grid, stream);
  }
}

}  // namespace

hipError_t launch_append_pages(const Geometry& g, const hkv_rope_axes* rope,
                               const int32_t* positions, int64_t axis_stride, const HeadView& q,
                               const HeadView& k, const HeadView& v, const HeadView& q_out,
                               int dtype, int32_t n_tokens, const int64_t* slots,
                               const PageView& dst, int dst_dtype, hipStream_t stream) {
  AppendPagesParams p;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.page_k = dst.k;
  p.page_v = dst.v;
  p.page = dst.page;
  p.token = dst.token;
  p.head = dst.head;
  p.slots = slots;
  p.n_slots = static_cast<int64_t>(g.n_blocks) * g.block_tokens;
  p.rcp_block = 1.0 / g.block_tokens;
  p.block_tokens = g.block_tokens;
  p.q_heads = q.n_heads;
  p.kv_heads = g.n_heads;
  p.vecs = q.n_heads + 2 * g.n_heads;
  p.positions = positions;
  p.axis_stride = axis_stride;
  for (int i = 0; i < kHeadDim / 2; ++i) {
    p.axis[i] = rope ? rope->axis[i] : -1;
    p.theta[i] = p.axis[i] < 0 ? 0.0 : quarter_turns(rope->rope_base, rope->freq[i]);
  }
  p.chunks = (p.vecs + kVecsPerWave - 1) / kVecsPerWave;
  p.waves = static_cast<int64_t>(n_tokens) * p.chunks;
  // a launch holds less than 2^32 threads: waves beyond 2^22 workgroups go round
  const int64_t need = (p.waves + kThreads / kWave - 1) / (kThreads / kWave);
  const dim3 grid(static_cast<unsigned>(need < (1 << 22) ? need : 1 << 22));
  const int pairs = rope ? rope->pairs : static_cast<int>(kHalfSplit);
  switch (dtype) {
    case kF32: return launch_source<kF32>(dst_dtype, pairs, p, grid, stream);
    case kF16: return launch_source<kF16>(dst_dtype, pairs, p, grid, stream);
    default: return launch_source<kBF16>(dst_dtype, pairs, p, grid, stream);
  }
}

}  // namespace hkv
