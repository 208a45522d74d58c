// Attention of queries over compressed records.
//
// One wave per (query row, query head), 8 lanes per cached vector, 8 tokens
// a step: each group of 8 lanes forms its token's score from the codes
// (scale and sm_scale applied in fp32), keeps its own running maximum, sum
// and weighted values, and the 8 groups are joined at the end.  Keys that
// moved by delta are met by the query turned by -delta: q . R(delta) k =
// R(-delta) q . k.
#include "rope_device.h"
#include "serve_launch.h"

namespace hkv {
namespace {

struct AttendParams {
  const uint8_t* rec;
  int64_t rec_block;
  int32_t n_blocks, block_tokens, n_heads, vecs;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* kv_len;
  const int32_t* q_start;
  int32_t max_len;
  int32_t max_queries;
  int32_t n_tokens;
  const char* q;
  char* out;
  int64_t q_token, q_head, o_token, o_head;
  int32_t q_heads, group;
  float* lse;
  float scale_log2;        // sm_scale * log2(e)
  int32_t causal;
  const int32_t* delta;
  double theta[kHeadDim / 2];
};

template <int FMT>
__device__ __forceinline__ void load_vector(const uint8_t* codes, int64_t v, int sub,
                                            float (&a)[8], float (&b)[8]) {
  if constexpr (FMT == kFP8) {
    const uint8_t* c = codes + v * kHeadDim + 8 * sub;
    fp8x8_to_f32(*reinterpret_cast<const u32x2*>(c), a);
    fp8x8_to_f32(*reinterpret_cast<const u32x2*>(c + 64), b);
  } else {
    const uint8_t* c = codes + v * (kHeadDim / 2) + 4 * sub;
    int4x8_to_f32(*reinterpret_cast<const uint32_t*>(c), a);
    int4x8_to_f32(*reinterpret_cast<const uint32_t*>(c + 32), b);
  }
}

template <int FMT, int DT, int PAIRS>
__global__ __launch_bounds__(kWave) void attend_kernel(AttendParams p) {
  constexpr int CB = FMT == kFP8 ? kHeadDim : kHeadDim / 2;
  constexpr int ES = ElemSize<DT>::value;
  const int lane = threadIdx.x;
  const int sub = lane & (kLanesPerVec - 1);
  const int grp = lane / kLanesPerVec;
  const int head = blockIdx.x % p.q_heads;
  const int j = blockIdx.x / p.q_heads;       // query of its request
  const int r = blockIdx.y;
  const int start = p.q_start ? min(max(p.q_start[r], 0), p.n_tokens) : r;
  const int end = p.q_start ? min(max(p.q_start[r + 1], 0), p.n_tokens) : r + 1;
  const int n_q = end - start;
  if (j >= n_q) return;
  const int len = min(max(p.kv_len[r], 0), p.max_len);
  const int64_t sees = p.causal ? min(static_cast<int64_t>(len) - n_q + j + 1,
                                      static_cast<int64_t>(len)) : len;
  const int64_t row = start + j;

  float qa[8], qb[8], ta[8], tb[8];
  const char* src = p.q + row * p.q_token + head * p.q_head + 8 * sub * ES;
  load8<DT>(src, qa);
  load8<DT>(src + 64 * ES, qb);
  int turned_by = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    ta[i] = qa[i];
    tb[i] = qb[i];
  }
  const int kh = head / p.group;
  float m = -INFINITY, l = 0.0f, oa[8] = {}, ob[8] = {};
  for (int64_t t0 = 0; t0 < sees; t0 += kVecsPerWave) {
    const int64_t t = t0 + grp;
    const bool in = t < sees;
    const int b = static_cast<int>((in ? t : sees - 1) / p.block_tokens);
    const int at = static_cast<int>((in ? t : sees - 1) - static_cast<int64_t>(b) * p.block_tokens);
    const int entry = p.table[r * p.table_stride + b];
    const bool live = in && entry >= 0 && entry < p.n_blocks;
    if (!live) continue;       // this group of lanes sits the step out
    if (p.delta) {
      const int d = p.delta[r * p.table_stride + b];
      if (d != turned_by) {
        float cs[8], sn[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ta[i] = qa[i];
          tb[i] = qb[i];
          cos_sin(d, p.theta[lane_pair(PAIRS, sub, i)], &cs[i], &sn[i]);
          sn[i] = -sn[i];
        }
        turn_runs<PAIRS>(ta, tb, cs, sn);
        turned_by = d;
      }
    }
    const uint8_t* rec = p.rec + entry * p.rec_block;
    const int v = at * p.n_heads + kh;
    const uint16_t* scales = reinterpret_cast<const uint16_t*>(rec + 2LL * p.vecs * CB);
    const float ks = f16_bits_to_f32(scales[v]);
    const float vs = f16_bits_to_f32(scales[static_cast<int64_t>(p.vecs) + v]);
    float a[8], c[8];
    load_vector<FMT>(rec, v, sub, a, c);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dot = __builtin_fmaf(a[i], ta[i], dot);
      dot = __builtin_fmaf(c[i], tb[i], dot);
    }
    dot += __shfl_xor(dot, 1, kLanesPerVec);
    dot += __shfl_xor(dot, 2, kLanesPerVec);
    dot += __shfl_xor(dot, 4, kLanesPerVec);
    const float s = dot * (ks * p.scale_log2);
    const float m_new = fmaxf(m, s);
    const float keep = m == m_new ? 1.0f : exp2f(m - m_new);
    const float w = exp2f(s - m_new);
    load_vector<FMT>(rec + static_cast<int64_t>(p.vecs) * CB, v, sub, a, c);
    l = l * keep + w;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      oa[i] = oa[i] * keep + w * vs * a[i];
      ob[i] = ob[i] * keep + w * vs * c[i];
    }
    m = m_new;
  }
#pragma unroll
  for (int off = kLanesPerVec; off < kWave; off <<= 1) {
    const float mo = __shfl_xor(m, off);
    const float m_new = fmaxf(m, mo);
    const float own = m == m_new ? 1.0f : exp2f(m - m_new);
    const float other = mo == m_new ? 1.0f : exp2f(mo - m_new);
    l = l * own + __shfl_xor(l, off) * other;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      oa[i] = oa[i] * own + __shfl_xor(oa[i], off) * other;
      ob[i] = ob[i] * own + __shfl_xor(ob[i], off) * other;
    }
    m = m_new;
  }
  const bool empty = l == 0.0f;
  const float inv = empty ? 0.0f : 1.0f / l;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    oa[i] *= inv;
    ob[i] *= inv;
  }
  if (grp == 0) {
    char* dst = p.out + row * p.o_token + head * p.o_head + 8 * sub * ES;
    store8<DT>(dst, oa);
    store8<DT>(dst + 64 * ES, ob);
    if (p.lse && sub == 0)
      p.lse[row * p.q_heads + head] =
          empty ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
  }
}

template <int FMT, int DT>
hipError_t launch_pairs(int pairs, const AttendParams& p, dim3 grid, hipStream_t stream) {
  if (pairs == kInterleaved)
    hipLaunchKernelGGL((attend_kernel<FMT, DT, kInterleaved>), grid, dim3(kWave), 0, stream, p);
  else
    hipLaunchKernelGGL((attend_kernel<FMT, DT, kHalfSplit>), grid, dim3(kWave), 0, stream, p);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_dtype(int dtype, int pairs, const AttendParams& p, dim3 grid, hipStream_t s) {
  switch (dtype) {
    case kF32: return launch_pairs<FMT, kF32>(pairs, p, grid, s);
    case kF16: return launch_pairs<FMT, kF16>(pairs, p, grid, s);
    default: return launch_pairs<FMT, kBF16>(pairs, p, grid, s);
  }
}

}  // namespace

int64_t attend_workspace_bytes(const Geometry&, const hkv_requests&, int32_t, int32_t, int) {
  return 0;
}

hipError_t launch_attend(const AttendCall& c, hipStream_t stream) {
  AttendParams p;
  p.rec = c.rec.base;
  p.rec_block = c.rec.block;
  p.n_blocks = c.g.n_blocks;
  p.block_tokens = c.g.block_tokens;
  p.n_heads = c.g.n_heads;
  p.vecs = c.g.vecs;
  p.table = c.req.block_table;
  p.table_stride = c.req.table_stride;
  p.kv_len = c.req.kv_len;
  p.q_start = c.req.q_start;
  p.max_len = c.req.max_blocks * c.g.block_tokens;
  p.max_queries = c.req.max_queries;
  p.n_tokens = c.n_tokens;
  p.q = c.q.data;
  p.out = c.out.data;
  p.q_token = c.q.token;
  p.q_head = c.q.head;
  p.o_token = c.out.token;
  p.o_head = c.out.head;
  p.q_heads = c.q.n_heads;
  p.group = c.q.n_heads / c.g.n_heads;
  p.lse = c.lse;
  p.scale_log2 = static_cast<float>(c.sm_scale * 1.44269504088896340736);
  p.causal = c.causal ? 1 : 0;
  p.delta = c.delta;
  for (int i = 0; i < kHeadDim / 2; ++i)
    p.theta[i] = c.delta ? quarter_turns(c.rope_base, i) : 0.0;
  const int32_t queries = c.req.max_queries < c.n_tokens ? c.req.max_queries : c.n_tokens;
  const dim3 grid(static_cast<unsigned>(queries) * c.q.n_heads,
                  static_cast<unsigned>(c.req.n_requests));
  return c.fmt == kFP8 ? launch_dtype<kFP8>(c.dtype, c.pairs, p, grid, stream)
                       : launch_dtype<kINT4>(c.dtype, c.pairs, p, grid, stream);
}

}  // namespace hkv
