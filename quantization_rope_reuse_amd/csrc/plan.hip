// Step plan: block tables, slots and positions from request lengths.
//
// Three prefix sums over the requests say where everything goes: q_start
// (new tokens), need (new blocks) and back (blocks of ended requests).  The
// free list is a stack, so the j-th new block of the step is entry
// top - 1 - j of the list after all pushes, and an entry at or above the old
// count is one that this call pushes: it is read from the ended request's
// table row, never from the list, so no workgroup waits for another.
//
// The work is a few bytes per request and token, so latency bounds it.
// Every workgroup therefore computes the three sums itself, in LDS, rather
// than waiting for a launch of its own to publish them: with at most 4,096
// requests that is at most 8 per thread and 32 KB read from L2.  The
// tokens, the pushed and the popped blocks are then spread over all threads
// of the grid, each finding its request by binary search in LDS.  48 decoding
// requests take 6 us, 1,500 requests with 40 prompts (62,000 tokens) 9.
#include "hkv_device.h"
#include "serve_launch.h"

namespace hkv {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWaves = kPlanThreads / kWave;
constexpr int kPerThread = kMaxStepRequests / kPlanThreads;   // requests per thread at most

struct PlanParams {
  hkv_step s;
  int32_t max_len;         // max_blocks * block_tokens
};

struct Sums {              // non-negative; q saturates at 2^31 - 1
  uint32_t q, need, back;
};

__device__ __forceinline__ Sums add(Sums a, Sums b) {
  return {min(a.q + b.q, 0x7FFFFFFFu), a.need + b.need, a.back + b.back};
}

struct Request {
  int len, held, n;        // cached tokens, blocks held, new tokens (negative: ends)
  bool fits;
  int need;
};

__device__ __forceinline__ Request request_of(const PlanParams& p, int r) {
  Request q;
  q.len = min(max(p.s.kv_len[r], 0), p.max_len);
  // len + block_tokens - 1 may pass 2^31: both terms are below it
  q.held = static_cast<int>((static_cast<uint32_t>(q.len) + (p.s.block_tokens - 1u)) /
                            static_cast<uint32_t>(p.s.block_tokens));
  q.n = p.s.new_tokens[r];
  q.fits = q.n <= p.max_len - q.len;
  const uint32_t want = static_cast<uint32_t>(q.len) + static_cast<uint32_t>(max(q.n, 0));
  q.need = q.n > 0 && q.fits
               ? static_cast<int>((want + (p.s.block_tokens - 1u)) / p.s.block_tokens) - q.held
               : 0;
  return q;
}

// Largest r with start[r] <= i, for start[0] = 0 <= i < start[n].
__device__ __forceinline__ int find(const uint32_t* start, int n, uint32_t i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanParams p) {
  extern __shared__ uint32_t lds[];
  const int n = p.s.n_requests;
  uint32_t* q_start = lds;                 // n + 1 entries each
  uint32_t* need = lds + (n + 1);
  uint32_t* back = lds + 2 * (n + 1);
  __shared__ Sums wave_sum[kPlanWaves];

  // Prefix sums: each thread its run of requests, then over the wave, then
  // over the waves.
  const int per = (n + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(static_cast<int>(threadIdx.x) * per, n);
  const int r1 = min(r0 + per, n);
  Sums own[kPerThread];
  Sums total = {0, 0, 0};
#pragma unroll
  for (int u = 0; u < kPerThread; ++u) {
    own[u] = {0, 0, 0};
    if (r0 + u < r1) {
      const Request q = request_of(p, r0 + u);
      own[u] = {static_cast<uint32_t>(max(q.n, 0)), static_cast<uint32_t>(q.need),
                static_cast<uint32_t>(q.n < 0 ? q.held : 0)};
      total = add(total, own[u]);
    }
  }
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  Sums run = total;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    Sums o = {static_cast<uint32_t>(__shfl_up(static_cast<int>(run.q), off)),
              static_cast<uint32_t>(__shfl_up(static_cast<int>(run.need), off)),
              static_cast<uint32_t>(__shfl_up(static_cast<int>(run.back), off))};
    if (lane >= off) run = add(run, o);
  }
  if (lane == kWave - 1) wave_sum[wave] = run;
  Sums before = {static_cast<uint32_t>(__shfl_up(static_cast<int>(run.q), 1)),
                 static_cast<uint32_t>(__shfl_up(static_cast<int>(run.need), 1)),
                 static_cast<uint32_t>(__shfl_up(static_cast<int>(run.back), 1))};
  if (lane == 0) before = {0, 0, 0};
  __syncthreads();
  Sums all = {0, 0, 0};
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    if (w == wave) before = add(all, before);
    all = add(all, wave_sum[w]);
  }
#pragma unroll
  for (int u = 0; u < kPerThread; ++u) {
    if (r0 + u < r1) {
      q_start[r0 + u] = before.q;
      need[r0 + u] = before.need;
      back[r0 + u] = before.back;
      before = add(before, own[u]);
    }
  }
  if (threadIdx.x == 0) {
    q_start[n] = all.q;
    need[n] = all.need;
    back[n] = all.back;
  }
  __syncthreads();

  const int cap = p.s.free_capacity;
  const int had = min(max(*p.s.free_count, 0), cap);
  const int top = static_cast<int>(
      min(static_cast<int64_t>(had) + static_cast<int64_t>(all.back), static_cast<int64_t>(cap)));

  // The entry of the list at i < top after all pushes, and the j-th pop.
  auto pushed = [&](uint32_t i) {
    const int r = find(back, n, i);
    return p.s.block_table[r * p.s.table_stride + (i - back[r])];
  };
  auto popped = [&](uint32_t j) {
    const int i = top - 1 - static_cast<int>(j);
    return i < had ? p.s.free_blocks[i] : pushed(static_cast<uint32_t>(i - had));
  };
  auto refused = [&](const Request& q, int r) {
    return q.n > 0 && (!q.fits || (q.need > 0 && need[r + 1] > static_cast<uint32_t>(top)));
  };

  const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;

  // Per request: its new length, start and flag; and the list's new count.
  // Refusals for lack of blocks hit every later request that needs one, so
  // the blocks taken are the needs of the requests before the first of them.
  for (int64_t r = first; r < n; r += step) {
    const Request q = request_of(p, static_cast<int>(r));
    const bool no = refused(q, static_cast<int>(r));
    p.s.kv_len_out[r] = q.n < 0 ? 0 : (no ? q.len : q.len + q.n);
    p.s.refused[r] = no ? 1 : 0;
    p.s.q_start[r] = static_cast<int32_t>(q_start[r]);
  }
  if (first == 0) {
    p.s.q_start[n] = static_cast<int32_t>(all.q);
    uint32_t taken = all.need;
    if (taken > static_cast<uint32_t>(top)) {
      // largest prefix of needs within the list
      int lo = 0, hi = n;                  // need[lo] <= top < need[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (need[mid] <= static_cast<uint32_t>(top))
          lo = mid;
        else
          hi = mid;
      }
      taken = need[lo];
    }
    *p.s.free_count_out = top - static_cast<int>(taken);
  }

  // Pushed blocks.
  for (int64_t i = first; i < top - had; i += step)
    p.s.free_blocks[had + i] = pushed(static_cast<uint32_t>(i));

  // Popped blocks: need is a prefix sum, so pop j belongs to request
  // find(need, j), whose requests are refused from the first that overruns.
  const int64_t pops = min(all.need, static_cast<uint32_t>(top));
  for (int64_t j = first; j < pops; j += step) {
    const int r = find(need, n, static_cast<uint32_t>(j));
    if (need[r + 1] > static_cast<uint32_t>(top)) continue;
    const int held = request_of(p, r).held;
    p.s.block_table[r * p.s.table_stride + held + (j - need[r])] = popped(static_cast<uint32_t>(j));
  }

  // Tokens.
  for (int64_t i = first; i < p.s.n_tokens; i += step) {
    int pos = 0;
    int64_t slot = -1;
    if (i < all.q) {
      const int r = find(q_start, n, static_cast<uint32_t>(i));
      const Request q = request_of(p, r);
      // a token of a refused request may stand beyond every position: clamp
      pos = static_cast<int>(min(static_cast<int64_t>(q.len) + (i - q_start[r]),
                                 static_cast<int64_t>(0x7FFFFFFF)));
      if (!refused(q, r)) {
        const int b = pos / p.s.block_tokens;
        const int entry = b < q.held ? p.s.block_table[r * p.s.table_stride + b]
                                     : popped(need[r] + static_cast<uint32_t>(b - q.held));
        if (entry >= 0)
          slot = static_cast<int64_t>(entry) * p.s.block_tokens + (pos - b * p.s.block_tokens);
      }
    }
    p.s.positions[i] = pos;
    p.s.slots[i] = slot;
  }
}

}  // namespace

hipError_t launch_plan(const hkv_step& s, hipStream_t stream) {
  PlanParams p;
  p.s = s;
  p.max_len = s.max_blocks * s.block_tokens;
  // One item per thread up to 256 workgroups.
  const int64_t items = s.n_tokens > s.n_requests ? s.n_tokens : s.n_requests;
  int64_t wgs = (items + kPlanThreads - 1) / kPlanThreads;
  wgs = wgs < 1 ? 1 : (wgs > 256 ? 256 : wgs);
  const size_t bytes = 3 * (static_cast<size_t>(s.n_requests) + 1) * sizeof(uint32_t);
  hipLaunchKernelGGL(plan_kernel, dim3(static_cast<unsigned>(wgs)), dim3(kPlanThreads), bytes,
                     stream, p);
  return hipGetLastError();
}

}  // namespace hkv
