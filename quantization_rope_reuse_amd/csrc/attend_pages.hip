// Attention over pages: how the work is shared out, and the join of partial
// results.
#include "attend_pages.h"
#include "attend_pages_share.h"

namespace hkv {
namespace {

// One workgroup per row that more than one range worked on: its waves (up to
// 8, by how many partial results a row may have) take the partial results in
// turn, a lane two dims; then the waves join in order.  Partial outputs are
// divided by their sums, so that no product here leaves their range.
constexpr int kJoinMost = 8;

__global__ __launch_bounds__(kJoinMost * kWave) void page_join_kernel(PageAttendParams p, int elem, int waves) {
  const int r = blockIdx.y;
  const PageSpan s = page_span(p, r);
  const int j = blockIdx.x / p.q_heads;
  if (j >= min(s.n_q, p.max_queries)) return;
  const int head = blockIdx.x - j * p.q_heads;
  const int kh = head / p.group;
  // The partial results of this row, w0 .. w1: of the ranges that its item
  // reaches over (one alone wrote the result), or the chunk kernel's cuts.
  int w0 = 0, w1 = p.splits - 1;
  uint32_t f0 = 0, per = 0;
  int in_item = 0;
  if (p.splits == 0) {
    const int row = j * p.group + (head - kh * p.group);
    const int item = row / kItemRows;
    const uint32_t first = p.prefix_out[r];
    const uint32_t tiles = (p.prefix_out[r + 1] - first) / ((s.rows + kItemRows - 1) / kItemRows);
    f0 = first + item * tiles;
    per = p.prefix_out[p.n_requests + 1];
    w0 = f0 / per;
    w1 = (f0 + tiles - 1) / per;
    if (w0 == w1) return;
    in_item = row - item * kItemRows;
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
  float2 o = make_float2(0.0f, 0.0f);      // divided by l
  for (int w = w0 + wave; w <= w1; w += waves) {
    const int64_t i = at(w);
    const float2 ml = p.part_ml[i];
    const float2 x = reinterpret_cast<const float2*>(p.part_o + i * kHeadDim)[lane];
    const float top = fmaxf(m, ml.x);
    const float keep = l * (m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top));
    const float more = ml.y * (ml.x == top ? 1.0f : __builtin_amdgcn_exp2f(ml.x - top));
    const float sum = keep + more;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const float a = keep * inv, b = more * inv;
    o.x = (keep == 0.0f ? 0.0f : a * o.x) + (more == 0.0f ? 0.0f : b * x.x);
    o.y = (keep == 0.0f ? 0.0f : a * o.y) + (more == 0.0f ? 0.0f : b * x.y);
    m = top;
    l = sum;
  }
  __shared__ float2 join_ml[kJoinMost];
  __shared__ float2 join_o[kJoinMost][kWave];
  join_o[wave][lane] = o;
  if (lane == 0) join_ml[wave] = make_float2(m, l);
  __syncthreads();
  if (threadIdx.x >= kHeadDim / 8) return;     // 8 dims a lane
  float top = kNoReference, sum = 0.0f, y[8] = {};
  for (int w = 0; w < waves; ++w) top = fmaxf(top, join_ml[w].x);
  for (int w = 0; w < waves; ++w)
    sum += join_ml[w].y * (join_ml[w].x == top ? 1.0f : __builtin_amdgcn_exp2f(join_ml[w].x - top));
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  for (int w = 0; w < waves; ++w) {
    const float f = join_ml[w].y * (join_ml[w].x == top ? 1.0f : __builtin_amdgcn_exp2f(join_ml[w].x - top)) * inv;
    if (f == 0.0f) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = join_o[w][4 * threadIdx.x + i];
      y[2 * i] += a.x * f;
      y[2 * i + 1] += a.y * f;
    }
  }
  const int64_t query = s.start + j;
  char* dst = p.out + query * p.o_token + head * p.o_head + 8 * threadIdx.x * elem;
  if (elem == 4)
    store8<kF32>(dst, y);
  else if (p.f16)
    store8<kF16>(dst, y);
  else
    store8<kBF16>(dst, y);
  if (p.lse && threadIdx.x == 0) p.lse[query * p.q_heads + head] = lse_of(top, sum);
}

}  // namespace

int64_t attend_pages_workspace_bytes(const Geometry& g, const hkv_requests& req, int32_t n_tokens,
                                     int32_t n_q_heads, int dtype) {
  return page_share_bytes(page_share_of(g, req, n_tokens, n_q_heads, dtype), req);
}

hipError_t launch_attend_pages(const PageAttendCall& c, hipStream_t stream) {
  PageAttendParams p = {};
  p.k = c.pages.k;
  p.v = c.pages.v;
  p.page = c.pages.page;
  p.token = c.pages.token;
  p.head = c.pages.head;
  p.num_pages = c.g.n_blocks;
  p.block_tokens = c.g.block_tokens;
  p.n_heads = c.g.n_heads;
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
  // a pool of no pages has no cached tokens
  p.max_len = c.g.n_blocks > 0 ? c.req.max_blocks * c.g.block_tokens : 0;
  p.max_queries = c.req.max_queries;
  p.n_tokens = c.n_tokens;
  p.f16 = c.dtype == HKV_F16;
  p.q = c.q.data;
  p.out = c.out.data;
  p.q_token = c.q.token;
  p.q_head = c.q.head;
  p.o_token = c.out.token;
  p.o_head = c.out.head;
  p.q_heads = c.q.n_heads;
  p.group = c.q.n_heads / c.g.n_heads;
  p.lse = c.lse;
  // |scale|; its sign and a scale of 0 go to the queries' bits
  const double scale = c.scores.sm_scale < 0 ? -c.scores.sm_scale : c.scores.sm_scale;
  constexpr double kLog2e = 1.44269504088896340736;
  p.scale = static_cast<float>(c.scores.cap > 0 ? scale / c.scores.cap : scale * kLog2e);
  p.cap_log2 = static_cast<float>(c.scores.cap * kLog2e);
  p.q_keep = p.scale > 0.0f ? ~0u : 0u;
  p.q_flip = c.scores.sm_scale < 0 ? (c.dtype == HKV_F32 ? 0x80000000u : 0x80008000u) : 0u;
  if (p.scale == 0.0f) p.scale = 1.0f;
  p.slopes = c.scores.slopes;
  p.causal = c.scores.causal != 0;
  p.window = c.scores.window;
  p.positions = c.scores.positions;
  p.begin = c.scores.begin;
  p.prefix = c.scores.prefix_len;

  const PageShare share = page_share_of(c.g, c.req, c.n_tokens, c.q.n_heads, c.dtype);
  p.splits = share.splits;
  p.ranges = share.ranges;
  p.min_tiles = share.min_tiles;
  p.part_rows = share.part_rows;
  if (share.rows > 0) {
    char* ws = static_cast<char*>(c.workspace);
    p.prefix_out = reinterpret_cast<uint32_t*>(ws);
    ws += page_prefix_bytes(c.req);
    p.part_ml = reinterpret_cast<float2*>(ws);
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
    e = c.dtype == HKV_F32   ? launch_page_chunk_f32(p, grid, stream)
        : c.dtype == HKV_F16 ? launch_page_chunk_f16(p, grid, stream)
                             : launch_page_chunk_bf16(p, grid, stream);
  } else {
    const dim3 grid = share.ranges > 0 ? dim3(static_cast<unsigned>(share.ranges * c.g.n_heads))
                                       : per_request(c.g.n_heads);
    e = c.dtype == HKV_F32   ? launch_page_rows_f32(p, grid, stream)
        : c.dtype == HKV_F16 ? launch_page_rows_f16(p, grid, stream)
                             : launch_page_rows_bf16(p, grid, stream);
  }
  if (e != hipSuccess || share.rows == 0) return e;
  const int64_t queries = c.req.max_queries < c.n_tokens ? c.req.max_queries : c.n_tokens;
  // about 8 partial results of a row for each wave
  const int64_t parts = share.splits > 0
                            ? share.splits
                            : share.ranges / (static_cast<int64_t>(c.req.n_requests) * share.items);
  int waves = 1;
  while (waves < kJoinMost && waves * 8 < parts) waves *= 2;
  hipLaunchKernelGGL(page_join_kernel,
                     dim3(static_cast<unsigned>(queries * c.q.n_heads),
                          static_cast<unsigned>(c.req.n_requests)),
                     dim3(waves * kWave), 0, stream, p, element_size(c.dtype), waves);
  return hipGetLastError();
}

}  // namespace hkv
