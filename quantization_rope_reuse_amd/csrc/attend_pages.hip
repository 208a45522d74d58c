// Attention over pages: how the work is shared out, and the join of partial
// results.
#include "attend_pages.h"
#include "attend_pages_share.h"

namespace hkv {
namespace {

// Joins the partial results of rows that more than one workgroup worked on.
// 16 lanes, 8 dims each, take a row's partial results in turn; where these are
// many, `sets` (1, 2, 4 .. 16) such lane groups take every sets-th of them and
// join in LDS, in order.  Partial outputs are divided by their sums, so that
// no product here leaves their range.
constexpr int kJoinThreads = 256;
constexpr int kJoinLanes = kHeadDim / 8;
constexpr int kJoinGroups = kJoinThreads / kJoinLanes;
static_assert(kJoinGroups == kJoinMostSets, "a workgroup's lane groups");

struct Joined {
  float m, l, o[8];                        // o divided by l
  __device__ __forceinline__ void add(float x_m, float x_l, const float (&x)[8]) {
    const float top = fmaxf(m, x_m);
    const float keep = l * (m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top));
    const float more = x_l * (x_m == top ? 1.0f : __builtin_amdgcn_exp2f(x_m - top));
    const float sum = keep + more;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const float a = keep * inv, b = more * inv;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (keep == 0.0f ? 0.0f : a * o[i]) + (more == 0.0f ? 0.0f : b * x[i]);
    m = top;
    l = sum;
  }
};

__global__ __launch_bounds__(kJoinThreads) void page_join_kernel(PageAttendParams p, int elem, int sets) {
  const int r = blockIdx.y;
  const int group = threadIdx.x / kJoinLanes, lane = threadIdx.x % kJoinLanes;
  const int set = group % sets;
  const PageSpan s = page_span(p, r);
  const int queries = min(s.n_q, p.max_queries);
  const int64_t row_head = static_cast<int64_t>(blockIdx.x) * (kJoinGroups / sets) + group / sets;
  const int j = static_cast<int>(row_head / p.q_heads);
  const int head = static_cast<int>(row_head - static_cast<int64_t>(j) * p.q_heads);
  const int kh = head / p.group;
  const int64_t query = s.start + j;
  // The partial results of this row, w0 .. w1: of the ranges that its item
  // reaches over, or the chunk kernel's cuts; where w0 = w1, that one wrote the
  // result.
  int w0 = 0, w1 = 0;
  uint32_t f0 = 0, per = 1;
  int in_item = 0;
  if (j < queries) {
    if (p.splits > 0) {
      w1 = p.part_n[query * p.q_heads + head] - 1;
    } else {
      const int row = j * p.group + (head - kh * p.group);
      const int item = row / kItemRows;
      const uint32_t first = p.prefix_out[r];
      const uint32_t tiles = (p.prefix_out[r + 1] - first) / ((s.rows + kItemRows - 1) / kItemRows);
      f0 = first + item * tiles;
      per = p.prefix_out[p.n_requests + 1];
      w0 = f0 / per;
      w1 = (f0 + tiles - 1) / per;
      in_item = row - item * kItemRows;
    }
  }
  auto at = [&](int w) {
    if (p.splits > 0) return (static_cast<int64_t>(w) * p.n_tokens + query) * p.q_heads + head;
    const int which = w == w0 && f0 > w0 * per ? 1 : 0;
    return (static_cast<int64_t>(w * 2 + which) * p.n_heads + kh) * p.part_rows + in_item;
  };
  Joined y = {kNoReference, 0.0f, {}};
  if (w0 < w1)
    for (int w = w0 + set; w <= w1; w += sets) {
      const int64_t i = at(w);
      const float2 ml = p.part_ml[i];
      const float4* o = reinterpret_cast<const float4*>(p.part_o + i * kHeadDim + 8 * lane);
      const float4 a = o[0], b = o[1];
      y.add(ml.x, ml.y, {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w});
    }
  if (sets > 1) {
    __shared__ float2 join_ml[kJoinGroups];
    __shared__ float join_o[kJoinGroups][kHeadDim];
    if (lane == 0) join_ml[group] = make_float2(y.m, y.l);
#pragma unroll
    for (int i = 0; i < 8; ++i) join_o[group][i * kJoinLanes + lane] = y.o[i];
    __syncthreads();
    if (set != 0 || w0 == w1) return;
    // all at once: no one waits for the one before it
    float top = kNoReference, sum = 0.0f;
    for (int w = 0; w < sets; ++w) top = fmaxf(top, join_ml[group + w].x);
    auto share = [&](int w) {
      const float2 ml = join_ml[group + w];
      return ml.y * (ml.x == top ? 1.0f : __builtin_amdgcn_exp2f(ml.x - top));
    };
    for (int w = 0; w < sets; ++w) sum += share(w);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    y = {top, sum, {}};
    for (int w = 0; w < sets; ++w) {
      const float f = share(w) * inv;
      if (f == 0.0f) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) y.o[i] += f * join_o[group + w][i * kJoinLanes + lane];
    }
  }
  if (w0 == w1) return;
  char* dst = p.out + query * p.o_token + head * p.o_head + 8 * lane * elem;
  if (elem == 4)
    store8<kF32>(dst, y.o);
  else if (p.f16)
    store8<kF16>(dst, y.o);
  else
    store8<kBF16>(dst, y.o);
  if (p.lse && lane == 0) p.lse[query * p.q_heads + head] = lse_of(y.m, y.l);
}

}  // namespace

int64_t attend_pages_workspace_bytes(const Geometry& g, const hkv_requests& req, int32_t n_tokens,
                                     int32_t n_q_heads, int dtype) {
  (void)dtype;
  const int64_t even = page_share_bytes(page_share_of(g, req, n_tokens, n_q_heads, false));
  const int64_t slanted = page_share_bytes(page_share_of(g, req, n_tokens, n_q_heads, true));
  return even > slanted ? even : slanted;
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
  const int together = c.dtype == HKV_F32 ? Group<kF32>::kTokens : Group<kBF16>::kTokens;
  p.grouped = c.g.block_tokens % together == 0 && c.pages.token < (int64_t{1} << 31) / 16;
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

  // rows that see very different numbers of tokens
  const bool slanted = p.causal && p.window == 0 && !p.begin &&
                       (p.positions || static_cast<int64_t>(p.max_queries) * 2 > p.max_len);
  const PageShare share = page_share_of(c.g, c.req, c.n_tokens, c.q.n_heads, slanted);
  p.splits = share.splits;
  p.ranges = share.ranges;
  p.min_tiles = share.min_tiles;
  p.part_rows = share.part_rows;
  if (share.rows > 0) {
    char* ws = static_cast<char*>(c.workspace);
    if (share.splits > 0)
      p.part_n = reinterpret_cast<int32_t*>(ws);
    else
      p.prefix_out = reinterpret_cast<uint32_t*>(ws);
    ws += share.index_bytes;
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
  const int sets = page_join_sets(share, c.req.n_requests);
  const int64_t rows_each = kJoinGroups / sets;
  hipLaunchKernelGGL(page_join_kernel,
                     dim3(static_cast<unsigned>((queries * c.q.n_heads + rows_each - 1) / rows_each),
                          static_cast<unsigned>(c.req.n_requests)),
                     dim3(kJoinThreads), 0, stream, p, element_size(c.dtype), sets);
  return hipGetLastError();
}

}  // namespace hkv
