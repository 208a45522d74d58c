// Append: new tokens' keys and values quantized into their slots of a pool
// of records.
//
// The quantizer of the put (quant_device.h), 8 lanes per vector; a vector is
// one (token, head) of K or V and finds its own record through its token's
// slot.  It reads a vector and writes its codes and scale, so bytes bound it:
// 32,777 tokens of 8 heads, fp16 to INT4, take 37 us, 4.6 TB/s of the 6.2 that
// a large elementwise pass reaches (from call to call 40, 4.2 TB/s; to FP8 43,
// 4.8; from fp32 60 and 64, 5.1 and 5.3); 96 tokens, one launch's latency, 3.
#include "quant_device.h"
#include "serve_launch.h"

namespace hkv {
namespace {

struct AppendParams {
  const char* k;
  const char* v;
  int64_t k_token, k_head, v_token, v_head;
  uint8_t* rec;
  int64_t rec_block;
  const int64_t* slots;
  int64_t n_slots;         // n_blocks * block_tokens
  double rcp_block;        // 1 / block_tokens
  double rcp_heads;        // 1 / n_heads
  int32_t block_tokens;
  int32_t n_heads;
  int32_t vecs;            // vectors of a record
  int64_t n_vecs;          // n_tokens * n_heads
};

// Quotient of v / d for 0 <= v < 2^52, given rcp = 1 / d in double: the
// product is off by less than one, so one step either way makes it exact.
__device__ __forceinline__ int64_t divide(int64_t v, int32_t d, double rcp) {
  int64_t q = static_cast<int64_t>(static_cast<double>(v) * rcp);
  const int64_t r = v - q * d;
  if (r < 0) --q;
  if (r >= d) ++q;
  return q;
}

template <int FMT, int SDT>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendParams p) {
  constexpr int CB = FMT == kFP8 ? kHeadDim : kHeadDim / 2;
  constexpr int ES = ElemSize<SDT>::value;
  const int lane = threadIdx.x & (kWave - 1);
  const int sub = lane & (kLanesPerVec - 1);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / kWave);
  for (int64_t wave = static_cast<int64_t>(blockIdx.x) * (kThreads / kWave) + threadIdx.x / kWave;
       wave * kVecsPerWave < p.n_vecs; wave += step) {
    const int64_t v = wave * kVecsPerWave + lane / kLanesPerVec;
    const int64_t vc = v < p.n_vecs ? v : p.n_vecs - 1;     // lanes past the end repeat the last
    const int kv = blockIdx.y;
    const int64_t t = divide(vc, p.n_heads, p.rcp_heads);
    const int h = static_cast<int>(vc - t * p.n_heads);
    const int64_t slot = p.slots[t];
    const bool active = v < p.n_vecs && slot >= 0 && slot < p.n_slots;
    const char* src = (kv ? p.v + t * p.v_token + h * p.v_head : p.k + t * p.k_token + h * p.k_head) +
                      8 * sub * ES;
    const RawSrc<SDT> ra = load_run<SDT>(src);
    const RawSrc<SDT> rb = load_run<SDT>(src + 64 * ES);
    const int64_t s = active ? slot : 0;
    const int64_t blk = divide(s, p.block_tokens, p.rcp_block);
    const int at = static_cast<int>(s - blk * p.block_tokens) * p.n_heads + h;
    uint8_t* rec = p.rec + blk * p.rec_block;
    float a[8], b[8];
    run_to_f32<SDT>(ra, a);
    run_to_f32<SDT>(rb, b);
    const uint32_t sbits = quant_vector<FMT, false>(
        a, b, rec + (static_cast<int64_t>(kv) * p.vecs + at) * CB, sub, active, nullptr);
    if (active && sub == 0)
      reinterpret_cast<uint16_t*>(rec + 2LL * p.vecs * CB)[static_cast<int64_t>(kv) * p.vecs + at] =
          static_cast<uint16_t>(sbits);
  }
}

template <int FMT>
hipError_t launch_fmt(int dtype, const AppendParams& p, dim3 grid, hipStream_t stream) {
  switch (dtype) {
    case kF32:
      hipLaunchKernelGGL((append_kernel<FMT, kF32>), grid, dim3(kThreads), 0, stream, p);
      break;
    case kF16:
      hipLaunchKernelGGL((append_kernel<FMT, kF16>), grid, dim3(kThreads), 0, stream, p);
      break;
    default:
      hipLaunchKernelGGL((append_kernel<FMT, kBF16>), grid, dim3(kThreads), 0, stream, p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_append(int fmt, int dtype, const Geometry& g, const HeadView& k,
                         const HeadView& v, int32_t n_tokens, const int64_t* slots,
                         const RecordView& dst, hipStream_t stream) {
  AppendParams p;
  p.k = k.data;
  p.v = v.data;
  p.k_token = k.token;
  p.k_head = k.head;
  p.v_token = v.token;
  p.v_head = v.head;
  p.rec = dst.base;
  p.rec_block = dst.block;
  p.slots = slots;
  p.n_slots = static_cast<int64_t>(g.n_blocks) * g.block_tokens;
  p.rcp_block = 1.0 / g.block_tokens;
  p.rcp_heads = 1.0 / g.n_heads;
  p.block_tokens = g.block_tokens;
  p.n_heads = g.n_heads;
  p.vecs = g.vecs;
  p.n_vecs = static_cast<int64_t>(n_tokens) * g.n_heads;
  constexpr int64_t per_wg = kVecsPerWave * (kThreads / kWave);
  // a launch holds less than 2^32 threads: vectors beyond 2^22 workgroups go round
  const int64_t need = (p.n_vecs + per_wg - 1) / per_wg;
  const dim3 grid(static_cast<unsigned>(need < (1 << 22) ? need : 1 << 22), 2);
  return fmt == kFP8 ? launch_fmt<kFP8>(dtype, p, grid, stream)
                     : launch_fmt<kINT4>(dtype, p, grid, stream);
}

}  // namespace hkv
