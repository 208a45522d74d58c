// Attention over pages for few query rows per key head (decodes, drafts): each
// wave works on tiles of its own.
//
// An item is up to 32 rows of a key head.  The tiles of all items are dealt
// out evenly over ranges, about one workgroup of four waves per CU; a
// workgroup's waves take a range's tiles in turn and join in LDS, and what
// reaches over several ranges is joined by a second kernel.
//
// Keys and values come straight into LDS, one tile of each per wave: the next
// tile's keys set out as soon as the scores are made, its values behind the
// output, and no wave waits for another.  The waits set by hand let the one be under
// way beside the other.  The compiler's do not: it waits for all of a wave's loads
// before it uses a table entry that an earlier turn has loaded (so the next keys set
// out behind this tile's values) and before it loads the next one into the same
// register (so the next values set out behind the next keys).  What overlaps is the
// four waves.  Memory bounds it (fp32: the matrix instructions): loads of random
// 64-token pages into LDS reach 5.7 TB/s on this card; 32 requests of up to 8,192
// tokens (64 heads over 8, bf16, 473 MB) take 96 to 108 us, 4.4 to 4.9 TB/s, one of
// 65,519 53 (5.1), the rest those waits, setting out, and passing from a request to
// the next.  With two workgroups a CU the first take 117 us for 110, both with the
// join.
#pragma once

#include "attend_pages.h"

namespace hkv {

// How many tiles of a request the dealing counts for each item: what its rows
// may see, from what is quick to find.
__device__ __forceinline__ TileList dealt_tiles(const PageAttendParams& p, const PageSpan& s) {
  int lo = 0, hi = s.len;
  const int queries = min(s.n_q, p.max_queries);
  if ((p.window > 0 || p.begin || (p.positions && p.causal)) && queries <= 16) {
    lo = INT32_MAX;
    hi = 0;
    for (int j = 0; j < queries; ++j) {
      const Sight v = sight_of(p, s, j);
      if (v.hi <= v.lo) continue;
      lo = min(lo, v.lo);
      hi = max(hi, v.hi);
    }
    lo = min(lo, hi);
  } else if (p.window > 0 && !p.positions) {
    lo = min(sight_of(p, s, 0).lo, s.len);
    if (p.begin) lo = max(min(max(s.len - s.n_q, -1) - p.window + 1, s.len), 0);
  }
  TileList t = tiles_of_view(s.pre, lo, hi, kPageRowsTile);
  t.count = max(t.count, 1);               // rows that see nothing are written all the same
  return t;
}

// Tiles are dealt by the turns of a workgroup's waves: an item's last turn may
// have fewer tiles than waves.  (Ranges that begin inside a turn pass from an item
// to the next more often: five drafts over 900 tokens, two items, take 23 us so for
// 16, 16 requests of up to 4,096 with five each in fp32 78 for 70.)
__device__ __forceinline__ int in_turns(int tiles) {
  static_assert((kPageRowsWaves & (kPageRowsWaves - 1)) == 0, "a mask");
  return (tiles + kPageRowsWaves - 1) & ~(kPageRowsWaves - 1);
}

template <int DT>
struct PageRowsShared {
  char tile[kPageRowsWaves][2][kPageRowsTile * Row<DT>::kBytes];    // keys, values; then joined
  float2 ml[kPageRowsWaves][kWave];
  uint32_t wave_sum[kPageRowsWaves];
  uint32_t prefix[kMaxDealtRequests + 2];
};

template <int DT, bool CAP, bool BIAS>
__global__ __launch_bounds__(kPageRowsThreads) __attribute__((amdgpu_waves_per_eu(DT == kF32 ? 1 : 2, DT == kF32 ? 1 : 2)))
void page_rows_kernel(PageAttendParams p) {
  constexpr int ES = ElemSize<DT>::value;
  constexpr int PP = 2;
  using R = Row<DT>;
  constexpr int kLoads = kPageRowsTile / R::kPerWave;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  PageRowsShared<DT>& sh = *reinterpret_cast<PageRowsShared<DT>*>(lds);
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int q32 = lane & 31, h = lane >> 5;
  const int kh = blockIdx.x % p.n_heads;
  const int range = blockIdx.x / p.n_heads;
  const int64_t head_off = kh * p.head;
  const char* none = reinterpret_cast<const char*>(kZeros);
  char* keys = sh.tile[wave][0];
  char* values = sh.tile[wave][1];

  uint32_t at = 0, end = 0;            // dealt tiles
  int r = 0, item = range, items = 0;
  const int n = p.n_requests;
  const bool few = n <= kWave;         // a wave's lanes hold the requests' tiles
  uint32_t run = 0;                    // tiles up to and with this lane's request
  auto tiles_of = [&](int i) {
    const PageSpan s = page_span(p, i);
    return s.rows > 0 ? static_cast<uint32_t>((s.rows + kItemRows - 1) / kItemRows) * in_turns(dealt_tiles(p, s).count) : 0u;
  };
  // tiles before request i
  auto before = [&](int i) -> uint32_t {
    if (few) return i > 0 ? __builtin_amdgcn_readlane(run, i - 1) : 0;
    return __builtin_amdgcn_readfirstlane(sh.prefix[i]);
  };
  if (p.ranges > 0) {
    if (few) {
      // every wave for itself, without LDS or a barrier
      run = lane < n ? tiles_of(lane) : 0;
      if (n > 1) {
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
          const uint32_t x = __shfl_up(run, off);
          if (lane >= off) run += x;
        }
      }
    } else {
      const int per_thread = (n + kPageRowsThreads - 1) / kPageRowsThreads;
      const int r0 = min(static_cast<int>(threadIdx.x) * per_thread, n);
      const int r1 = min(r0 + per_thread, n);
      uint32_t sum = 0;
      for (int i = r0; i < r1; ++i) {
        const uint32_t x = tiles_of(i);
        sh.prefix[i + 1] = x;
        sum += x;
      }
      uint32_t upto = sum;
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const uint32_t x = __shfl_up(upto, off);
        if (lane >= off) upto += x;
      }
      if (lane == kWave - 1) sh.wave_sum[wave] = upto;
      __syncthreads();
      uint32_t sums = upto - sum;
      for (int w = 0; w < wave; ++w) sums += sh.wave_sum[w];
      for (int i = r0; i < r1; ++i) {
        sums += sh.prefix[i + 1];
        sh.prefix[i + 1] = sums;
      }
      if (threadIdx.x == 0) sh.prefix[0] = 0;
      __syncthreads();
    }
    const uint32_t total = before(n);
    const uint32_t per = in_turns(max((total + p.ranges - 1) / p.ranges, static_cast<uint32_t>(p.min_tiles)));
    if (blockIdx.x == 0) {
      if (few) {
        if (wave == 0 && lane < n) p.prefix_out[lane + 1] = run;
        if (threadIdx.x == 0) p.prefix_out[0] = 0;
      } else {
        for (int i = threadIdx.x; i <= n; i += kPageRowsThreads) p.prefix_out[i] = sh.prefix[i];
      }
      if (threadIdx.x == 0) p.prefix_out[n + 1] = per;
    }
    at = min(range * per, total);      // range * per < total + per * ranges: below 2^32
    end = min(at + per, total);
    if (at >= end) return;
    if (few) {
      r = __builtin_popcountll(__ballot(lane < n && run <= at));
    } else {
      int last = n;
      while (last - r > 1) {
        const int mid = (r + last) >> 1;
        if (before(mid) <= at)
          r = mid;
        else
          last = mid;
      }
    }
  } else {
    r = blockIdx.y;
    items = (page_span(p, r).rows + kItemRows - 1) / kItemRows;
  }

  const uint32_t first_at = at;
  while (p.ranges > 0 ? at < end : item < items) {
    // (requests without rows have no tiles)
    if (p.ranges > 0)
      while (before(r + 1) <= at) ++r;
    r = __builtin_amdgcn_readfirstlane(r);
    const PageSpan s = page_span(p, r);
    TileList list = dealt_tiles(p, s);     // (the same in all lanes: branches on it are scalar)
    list.pre = __builtin_amdgcn_readfirstlane(list.pre);
    list.lo = __builtin_amdgcn_readfirstlane(list.lo);
    list.count = __builtin_amdgcn_readfirstlane(list.count);
    int seg0 = 0, seg1 = list.count, dealt = 0;
    bool whole = true;
    if (p.ranges > 0) {
      const uint32_t in = at - before(r), tiles = in_turns(list.count);
      item = in / tiles;
      seg0 = in - item * tiles;
      dealt = min(tiles - seg0, end - at);
      seg1 = min(seg0 + dealt, list.count);
      whole = dealt == static_cast<int>(tiles);
    }
    const int32_t* table = p.table + r * p.table_stride;

    const int row = min(item * kItemRows + q32, s.rows - 1);
    const int j = row / p.group;
    const int head = kh * p.group + (row - j * p.group);
    const int64_t query = s.start + j;
    const char* q_row = p.q + query * p.q_token + head * p.q_head;
    Queries<DT> q;
    q.load(q_row, h, p.q_keep, p.q_flip);
    const Sight sight = sight_of(p, s, j);
    const View view = view_of_wave(sight);
    const ScoreScale f = scale_of<BIAS>(p, head);

    RowsState st;
#pragma unroll
    for (int d = 0; d < 4; ++d) st.o[d] = f32x16{};
    st.m = kNoReference;
    st.l = 0.0f;
    st.far = false;

    // Tiles to come: the table entry of this lane's token of one, the keys and
    // values of the one before.
    auto seen_from = [&](int i) {
      while (i < seg1 && !view.some(list.at(i) * kPageRowsTile, kPageRowsTile)) i += kPageRowsWaves;
      return i;
    };
    int entry = -1;
    auto entry_of = [&](int i) {
      const int token = list.at(i) * kPageRowsTile + q32;
      return token < s.len ? table[block_of(p, token)] : -1;
    };
    int64_t off[kLoads];
    uint32_t live_next = 0;
    // places of tile i's tokens, from their table entries
    auto place = [&](int i) __attribute__((always_inline)) {
      const int id = here(lane);
      const int token = list.at(i) * kPageRowsTile + q32;
      const bool known = token < s.len && static_cast<uint32_t>(entry) < static_cast<uint32_t>(p.num_pages);
      const int64_t at = known ? entry * p.page + (token - block_of(p, token) * p.block_tokens) * p.token + head_off
                               : int64_t{-1};
      live_next = static_cast<uint32_t>(__ballot(known));
#pragma unroll
      for (int n = 0; n < kLoads; ++n) off[n] = __shfl(at, R::kPerWave * n + id / R::kChunks);
    };
    auto bring_keys = [&](char* to) __attribute__((always_inline)) {
      const int id = here(lane);
#pragma unroll
      for (int n = 0; n < kLoads; ++n) {
        const int t = R::kPerWave * n + id / R::kChunks;
        bring16(off[n] < 0 ? none : p.k + off[n] + (R::key(t, id % R::kChunks) << 4), to + 16 * kWave * n);
      }
    };
    auto bring_values = [&](char* to) __attribute__((always_inline)) {
      const int id = here(lane);
#pragma unroll
      for (int n = 0; n < kLoads; ++n) {
        const int t = R::kPerWave * n + id / R::kChunks;
        bring16(off[n] < 0 ? none : p.v + off[n] + (R::value(t, id % R::kChunks) << 4), to + 16 * kWave * n);
      }
    };
    int i = seen_from(seg0 + wave);
    if (i < seg1) {
      entry = entry_of(i);
      place(i);
      bring_keys(keys);
      int next = seen_from(i + kPageRowsWaves);
      if (next < seg1) entry = entry_of(next);
      bring_values(values);
      // (the two areas do not overlap: reads of one need not wait for loads of the other)
      auto step = [&](char* __restrict__ k_area, char* __restrict__ v_area) __attribute__((always_inline)) {
        const uint32_t live = live_next;
        const int first = list.at(i) * kPageRowsTile;
        int after = seg1;
        wait_loads<kLoads>();              // the keys; the values need not be there
        f32x16 acc[1] = {score_tile<DT>(k_area, q, lane)};
        wait_loads<kLoads>();              // the keys are read
        if (next < seg1) {
          place(next);
          bring_keys(k_area);
          after = seen_from(next + kPageRowsWaves);
        }
        const bool part = live != ~0u || !view.all(first, kPageRowsTile);
        float from_first = 0.0f;
        if constexpr (BIAS) from_first = static_cast<float>(static_cast<double>(sight.pos) - (first + 4 * h));
        const uint64_t seen = part ? seen_of(sight, live, first, h) : 0;
        Weights<DT, PP> w[1];
        refer_tile<DT, CAP, BIAS, 1>(acc, scores_of<CAP, BIAS, 1>(acc, f, from_first), st, f, part, seen);
        st.l += weigh_tile<DT, PP>(acc[0], w[0], st);
        if (next < seg1)
          wait_loads<kLoads>();            // the values; the next keys need not be there
        else
          wait_loads<0>();
        output_tile<DT, PP>(v_area, w[0], st.o, lane);
        if (next < seg1) {
          wait_loads<kLoads>();            // the values are read
          if (after < seg1) entry = entry_of(after);     // (before them: it arrives first)
          bring_values(v_area);
        }
        i = next;
        next = after;
      };
      while (i < seg1) step(keys, values);
    }
    const WaveTiles mine = {list, seg0 + wave, seg1, kPageRowsWaves, kPageRowsTile};
    finish_rows<DT, PP, CAP, BIAS, 1>(p, table, head_off, q_row, sight, s.len, mine, st, f, lane);

    // The waves join: wave d takes dims 32 d ..
    const int last_lane = here(lane), last_q = last_lane & 31, last_h = last_lane >> 5;
    f32x4* mine_o = reinterpret_cast<f32x4*>(sh.tile[wave]);
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int a = 0; a < 4; ++a)
        mine_o[(4 * d + a) * kWave + last_lane] =
            f32x4{st.o[d][4 * a], st.o[d][4 * a + 1], st.o[d][4 * a + 2], st.o[d][4 * a + 3]};
    sh.ml[wave][last_lane] = make_float2(st.m, st.l);
    __syncthreads();
    float top = kNoReference;
#pragma unroll
    for (int w = 0; w < kPageRowsWaves; ++w) top = fmaxf(top, sh.ml[w][last_lane].x);
    float share[kPageRowsWaves], sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kPageRowsWaves; ++w) {
      const float2 ml = sh.ml[w][last_lane];
      share[w] = ml.y * (ml.x == top ? 1.0f : __builtin_amdgcn_exp2f(ml.x - top));
      sum += share[w];
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    float y[16] = {};
#pragma unroll
    for (int w = 0; w < kPageRowsWaves; ++w) {
      const float x = share[w] * inv;
      const f32x4* o = reinterpret_cast<const f32x4*>(sh.tile[w]);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const f32x4 z = o[(4 * wave + a) * kWave + last_lane];
#pragma unroll
        for (int b = 0; b < 4; ++b) y[4 * a + b] += x == 0.0f ? 0.0f : x * z[b];
      }
    }
    const int last_row = item * kItemRows + last_q;
    if (last_row < s.rows) {
      const int last_j = last_row / p.group;
      const int last_head = kh * p.group + (last_row - last_j * p.group);
      const int64_t last_query = s.start + last_j;
      const int64_t part_row =
          (static_cast<int64_t>(range * 2 + (at > first_at ? 1 : 0)) * p.n_heads + kh) * p.part_rows + last_q;
      char* dst = whole ? p.out + last_query * p.o_token + last_head * p.o_head
                        : reinterpret_cast<char*>(p.part_o + part_row * kHeadDim);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int dim = 32 * wave + 8 * a + 4 * last_h;
        const float z[4] = {y[4 * a], y[4 * a + 1], y[4 * a + 2], y[4 * a + 3]};
        if (whole)
          store4<DT>(dst + dim * ES, z);
        else
          store4<kF32>(dst + dim * 4, z);
      }
      if (wave == 0 && last_h == 0) {
        if (!whole)
          p.part_ml[part_row] = make_float2(top, sum);
        else if (p.lse)
          p.lse[last_query * p.q_heads + last_head] = lse_of(top, sum);
      }
    }
    __syncthreads();                     // the tiles' LDS is free
    if (p.ranges > 0)
      at += dealt;
    else
      item += gridDim.x / p.n_heads;
  }
}

template <int DT>
hipError_t launch_page_rows(const PageAttendParams& p, dim3 grid, hipStream_t stream) {
  constexpr int kBytes = sizeof(PageRowsShared<DT>);
  auto* kernel = p.cap_log2 > 0.0f ? (p.slopes ? page_rows_kernel<DT, true, true> : page_rows_kernel<DT, true, false>)
                                   : (p.slopes ? page_rows_kernel<DT, false, true> : page_rows_kernel<DT, false, false>);
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, grid, dim3(kPageRowsThreads), kBytes, stream, p);
  return hipGetLastError();
}

}  // namespace hkv
