// Attention of queries over compressed records: how the work is shared out,
// and the join of partial results.
#include "attend_rows.h"
#include "attend_share.h"

namespace hkv {
namespace {

// One workgroup per row that more than one range worked on: its waves (up to
// 8, by how many partial results a row may have) take the partial results in
// turn, a lane two dims; then the waves join in order.
constexpr int kJoinMost = 8;

__global__ __launch_bounds__(kJoinMost * kWave) void attend_join_kernel(AttendParams p, int item_rows,
                                                                        int waves) {
  const int r = blockIdx.y;
  const Span s = span_of(p, r);
  const int j = blockIdx.x / p.q_heads;
  if (j >= min(s.n_q, p.max_queries)) return;
  const int head = blockIdx.x - j * p.q_heads;
  const int kh = head / p.group;
  // The partial results of this row: w0 .. w1.  The rows kernel's ranges that
  // an item reaches over (alone, it wrote the result), or the prompt kernel's
  // cuts.
  int w0 = 0, w1 = p.splits - 1;
  uint32_t f0 = 0, per = 0;
  int64_t in_item = 0;
  if (p.splits == 0) {
    const int row = j * p.group + (head - kh * p.group);
    const int item = row / item_rows;
    const uint32_t tiles = tiles_of(s);
    f0 = p.prefix_out[r] + item * tiles;
    per = p.prefix_out[p.n_requests + 1];
    w0 = f0 / per;
    w1 = (f0 + tiles - 1) / per;
    if (w0 == w1) return;
    in_item = row - item * item_rows;
  }
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  auto at = [&](int w) {
    if (p.splits > 0)
      return (static_cast<int64_t>(w) * p.n_tokens + s.start + j) * p.q_heads + head;
    const int which = w == w0 && f0 > w0 * per ? 1 : 0;
    return (static_cast<int64_t>(w * 2 + which) * p.n_heads + kh) * p.part_rows + in_item;
  };
  float m = kNoReference, l = 0.0f;
  float2 o = make_float2(0.0f, 0.0f);
  constexpr int kBatch = 8;
  for (int w = w0 + wave; w <= w1; w += waves * kBatch) {
    float2 ml[kBatch], x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t i = at(min(w + u * waves, w1));
      ml[u] = reinterpret_cast<const float2*>(p.part_ml)[i];
      x[u] = reinterpret_cast<const float2*>(p.part_o + i * kHeadDim)[lane];
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (w + u * waves <= w1) top = fmaxf(top, ml[u].x);
    const float keep = m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
    l *= keep;
    o.x *= keep;
    o.y *= keep;
    m = top;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (w + u * waves > w1) break;
      const float f = ml[u].x == m ? 1.0f : __builtin_amdgcn_exp2f(ml[u].x - m);
      l += ml[u].y * f;
      o.x += x[u].x * f;
      o.y += x[u].y * f;
    }
  }
  __shared__ float2 join_ml[kJoinMost];
  __shared__ float2 join_o[kJoinMost][kWave];
  join_o[wave][lane] = o;
  if (lane == 0) join_ml[wave] = make_float2(m, l);
  __syncthreads();
  if (threadIdx.x >= kHeadDim / 8) return;     // 8 dims a lane
  float top = kNoReference, sum = 0.0f, y[8] = {};
  for (int w = 0; w < waves; ++w) top = fmaxf(top, join_ml[w].x);
  for (int w = 0; w < waves; ++w) {
    const float f = join_ml[w].x == top ? 1.0f : __builtin_amdgcn_exp2f(join_ml[w].x - top);
    sum += join_ml[w].y * f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = join_o[w][4 * threadIdx.x + i];
      y[2 * i] += a.x * f;
      y[2 * i + 1] += a.y * f;
    }
  }
  const bool empty = sum == 0.0f;
  const float inv = empty ? 0.0f : 1.0f / (sum * kWeightScale);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = empty ? 0.0f : y[i] * inv;
  const int64_t query = s.start + j;
  store8_any(p.dtype, p.out + query * p.o_token + head * p.o_head + 8 * threadIdx.x * p.elem, y);
  if (p.lse && threadIdx.x == 0)
    p.lse[query * p.q_heads + head] = log_sum(top, sum);
}

}  // namespace

int64_t attend_workspace_bytes(const Geometry& g, const hkv_requests& req, int32_t n_tokens,
                               int32_t n_q_heads, int dtype) {
  int64_t most = 0;
  for (int fmt : {HKV_FP8_E4M3, HKV_INT4})
    for (bool moved : {false, true}) {
      const int64_t b = share_bytes(share_of(fmt, moved, g, req, n_tokens, n_q_heads, dtype), req);
      most = b > most ? b : most;
    }
  return most;
}

hipError_t launch_attend(const AttendCall& c, hipStream_t stream) {
  AttendParams p;
  p.rec = c.rec.base;
  p.rec_block = c.rec.block;
  p.n_blocks = c.g.n_blocks;
  p.block_tokens = c.g.block_tokens;
  p.n_heads = c.g.n_heads;
  p.vecs = c.g.vecs;
  // ceil(2^(31 + s) / d) with 2^s >= d makes the quotient exact below 2^31
  int s = 0;
  while ((int64_t{1} << s) < c.g.block_tokens) ++s;
  p.block_shift = 31 + s;
  p.block_magic = ((uint64_t{1} << p.block_shift) + c.g.block_tokens - 1) / c.g.block_tokens;
  p.n_requests = c.req.n_requests;
  p.table = c.req.block_table;
  p.table_stride = c.req.table_stride;
  p.kv_len = c.req.kv_len;
  p.q_start = c.req.q_start;
  // a pool of no records has no cached tokens
  p.max_len = c.g.n_blocks > 0 ? c.req.max_blocks * c.g.block_tokens : 0;
  p.max_queries = c.req.max_queries;
  p.n_tokens = c.n_tokens;
  p.dtype = c.dtype;
  p.elem = element_size(c.dtype);
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
  p.pairs = c.pairs;
  for (int i = 0; i < kHeadDim / 2; ++i)
    p.theta[i] = c.delta ? quarter_turns(c.rope_base, i) : 0.0;

  const Share share = share_of(c.fmt, c.delta != nullptr, c.g, c.req, c.n_tokens, c.q.n_heads, c.dtype);
  p.splits = share.splits;
  p.set_heads = share.set_heads;
  p.head_sets = share.head_sets;
  p.ranges = share.ranges;
  p.min_tiles = share.min_tiles;
  p.part_rows = share.part_rows;
  p.prefix_out = nullptr;
  p.part_ml = nullptr;
  p.part_o = nullptr;
  if (share.rows > 0) {
    char* ws = static_cast<char*>(c.workspace);
    p.prefix_out = reinterpret_cast<uint32_t*>(ws);
    ws += prefix_bytes(c.req);
    p.part_ml = reinterpret_cast<float*>(ws);
    p.part_o = reinterpret_cast<float*>(ws + (share.rows * 8 + 15) / 16 * 16);
  }
  // items beyond 65,535 workgroups per request are taken in turn
  auto per_request = [&](int64_t sets) {
    const int64_t most = 65535 / sets;
    int64_t x = share.items < most ? share.items : most;
    x = x < 1 ? 1 : x;
    return dim3(static_cast<unsigned>(x * sets), static_cast<unsigned>(c.req.n_requests));
  };
  hipError_t e;
  if (share.splits > 0) {
    const dim3 grid = per_request(static_cast<int64_t>(c.g.n_heads) * share.splits);
    e = c.fmt == kFP8 ? launch_prompt_fp8(p, grid, stream) : launch_prompt_int4(p, grid, stream);
  } else {
    // at most 44 KB of LDS (the prefix sums of kMaxFlatRequests requests: 4)
    size_t bytes = kRowsWaves * kWaveAreaBytes + (kRowsWaves / 2) * share.nt * (8192 + 512);
    if (share.ranges > 0) bytes += static_cast<size_t>(prefix_bytes(c.req));
    const dim3 grid = share.ranges > 0 ? dim3(static_cast<unsigned>(share.ranges * share.head_sets))
                                       : per_request(share.head_sets);
    e = c.fmt == kFP8 ? launch_rows_fp8(p, share.hp, share.nt, grid, bytes, stream)
                      : launch_rows_int4(p, share.hp, share.nt, grid, bytes, stream);
  }
  if (e != hipSuccess || share.rows == 0) return e;
  const int64_t queries = c.req.max_queries < c.n_tokens ? c.req.max_queries : c.n_tokens;
  // about 8 partial results of a row for each wave
  const int64_t parts = share.splits > 0
                            ? share.splits
                            : share.ranges / (static_cast<int64_t>(c.req.n_requests) * share.items);
  int waves = 1;
  while (waves < kJoinMost && waves * 8 < parts) waves *= 2;
  hipLaunchKernelGGL(attend_join_kernel,
                     dim3(static_cast<unsigned>(queries * c.q.n_heads),
                          static_cast<unsigned>(c.req.n_requests)),
                     dim3(waves * kWave), 0, stream, p, 16 * share.nt / share.hp, waves);
  return hipGetLastError();
}

}  // namespace hkv
