// Attention over pages for many query rows per key head (chunks of prompts,
// rows picked for recomputing).
//
// A workgroup of 8 waves takes 256 rows of a key head, 32 a wave, and walks the
// tokens that some of them see in tiles of 64, which all waves bring into LDS
// together and each uses for its own rows; tiles are cut into ranges where
// items are too few for the CUs.  The loads of the tiles to come are under way
// while a tile is worked on; one barrier a tile.
#pragma once

#include "attend_pages.h"

namespace hkv {

template <int DT> constexpr int kRing = DT == kF32 ? 2 : 3;      // tiles in LDS

template <int DT>
struct PageChunkShared {
  char tile[kRing<DT>][2][kPageChunkTile * Row<DT>::kBytes];     // keys, values
  uint64_t live[kRing<DT>];            // tokens of the tile that exist
  int bounds[kPageChunkWaves][3];
};

template <int DT, bool CAP, bool BIAS>
__global__ __launch_bounds__(kPageChunkThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void page_chunk_kernel(PageAttendParams p) {
  constexpr int ES = ElemSize<DT>::value;
  constexpr int N = kPageChunkTile / kSub;
  using R = Row<DT>;
  constexpr int kRows = kPageChunkTile / kPageChunkWaves;        // that a wave brings
  constexpr int kLoads = kRows / R::kPerWave;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  PageChunkShared<DT>& sh = *reinterpret_cast<PageChunkShared<DT>*>(lds);
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int q32 = lane & 31, h = lane >> 5;
  const char* none = reinterpret_cast<const char*>(kZeros);

  const int kh = blockIdx.x % p.n_heads;
  const int rest = blockIdx.x / p.n_heads;
  const int split = rest % p.splits;
  const int r = blockIdx.y;
  const PageSpan s = page_span(p, r);
  const int row_tiles = (s.rows + kPageChunkRows - 1) / kPageChunkRows;
  const int step_items = gridDim.x / (p.n_heads * p.splits);
  const int64_t head_off = kh * p.head;
  const int32_t* table = p.table + r * p.table_stride;

  // Later rows see more: they come first.
  for (int back = rest / p.splits; back < row_tiles; back += step_items) {
    const int row0 = (row_tiles - 1 - back) * kPageChunkRows;
    const int row = min(row0 + kItemRows * wave + q32, s.rows - 1);
    const int j = row / p.group;
    const int head = kh * p.group + (row - j * p.group);
    const int64_t query = s.start + j;
    const char* q_row = p.q + query * p.q_token + head * p.q_head;
    const Sight sight = sight_of(p, s, j);
    const View view = view_of_wave(sight);
    const ScoreScale f = scale_of<BIAS>(p, head);
    Queries<DT> q;
    q.load(q_row, h, p.q_keep, p.q_flip);
    __syncthreads();                       // the last rows' LDS is free
    if (lane == 0) {
      sh.bounds[wave][0] = view.pre_most;
      sh.bounds[wave][1] = view.lo_least;
      sh.bounds[wave][2] = view.hi_most;
    }
    __syncthreads();
    int pre = 0, lo = INT32_MAX, hi = 0;
#pragma unroll
    for (int w = 0; w < kPageChunkWaves; ++w) {
      pre = max(pre, sh.bounds[w][0]);
      lo = min(lo, sh.bounds[w][1]);
      hi = max(hi, sh.bounds[w][2]);
    }
    pre = __builtin_amdgcn_readfirstlane(pre);
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    const TileList list = tiles_of_view(pre, lo, hi, kPageChunkTile);
    const int per = (list.count + p.splits - 1) / p.splits;
    const int t0 = min(split * per, list.count);
    const int t1 = min(t0 + per, list.count);

    RowsState st;
#pragma unroll
    for (int d = 0; d < 4; ++d) st.o[d] = f32x16{};
    st.m = kNoReference;
    st.l = 0.0f;
    st.far = false;

    int entry = -1;
    auto entry_of = [&](int t) __attribute__((always_inline)) {
      const int token = list.at(t) * kPageChunkTile + kRows * wave + (here(lane) & (kRows - 1));
      return token < s.len ? table[block_of(p, token)] : -1;
    };
    // Tile t into `area`, from its table entries; and tile t + 1's entries set out.
    auto bring = [&](int t, char* area, uint64_t* live) __attribute__((always_inline)) {
      const int id = here(lane);
      const int token = list.at(t) * kPageChunkTile + kRows * wave + (id & (kRows - 1));
      const bool known = token < s.len && static_cast<uint32_t>(entry) < static_cast<uint32_t>(p.num_pages);
      const int64_t at = known ? entry * p.page + (token - block_of(p, token) * p.block_tokens) * p.token + head_off
                               : int64_t{-1};
      const uint64_t alive = __ballot(known);
      if (id == 0) reinterpret_cast<uint8_t*>(live)[wave] = static_cast<uint8_t>(alive);
      if (t + 1 < t1) entry = entry_of(t + 1);
#pragma unroll
      for (int n = 0; n < kLoads; ++n) {
        const int first = R::kPerWave * n + id / R::kChunks;
        const int64_t off = __shfl(at, first);
        const int to = kRows * wave + first;
        char* keys = area + kRows * R::kBytes * wave + 16 * kWave * n;
        char* values = keys + kPageChunkTile * R::kBytes;
        bring16(off < 0 ? none : p.k + off + (R::key(to, id % R::kChunks) << 4), keys);
        bring16(off < 0 ? none : p.v + off + (R::value(to, id % R::kChunks) << 4), values);
      }
    };
    auto work = [&](const char* tile, const uint64_t* live_at, int first) __attribute__((always_inline)) {
      if (!view.some(first, kPageChunkTile)) return;
      const uint64_t live = *live_at;
      const uint64_t alive = static_cast<uint64_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(live >> 32))) << 32 |
                             static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(live)));
      f32x16 acc[N];
#pragma unroll
      for (int u = 0; u < N; ++u) acc[u] = score_tile<DT>(tile + u * kSub * R::kBytes, q, lane);
      const bool part = alive != ~uint64_t{0} || !view.all(first, kPageChunkTile);
      float from_first = 0.0f;
      if constexpr (BIAS) from_first = static_cast<float>(static_cast<double>(sight.pos) - (first + 4 * h));
      const uint64_t seen = part ? seen_of(sight, alive, first, h) : 0;
      Weights<DT, 1> w[N];
      weigh_tile<DT, 1, CAP, BIAS, N>(acc, w, st, f, from_first, part, seen);
#pragma unroll
      for (int u = 0; u < N; ++u)
        output_tile<DT, 1>(tile + (kPageChunkTile + u * kSub) * R::kBytes, w[u], st.o, lane);
    };
    // (the areas do not overlap: reads of one need not wait for loads of another)
    auto step = [&](int t, const char* __restrict__ now, const uint64_t* __restrict__ now_live,
                    char* __restrict__ next, uint64_t* __restrict__ next_live) __attribute__((always_inline)) {
      if (t + kRing<DT> - 1 < t1) bring(t + kRing<DT> - 1, next, next_live);
      work(now, now_live, list.at(t) * kPageChunkTile);
    };
    if (t0 < t1) {
      entry = entry_of(t0);
#pragma unroll
      for (int n = 0; n < kRing<DT> - 1; ++n)
        if (t0 + n < t1) bring(t0 + n, sh.tile[n][0], &sh.live[n]);
      int slot = 0;
      for (int t = t0; t < t1; ++t) {
        // this tile's loads; the next ones' may be under way (a ring of two has none)
        if (kRing<DT> > 2 && t + 1 < t1)
          wait_loads<2 * kLoads*(kRing<DT> - 2)>();
        else
          wait_loads<0>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const int free_slot = slot == 0 ? kRing<DT> - 1 : slot - 1;
        step(t, sh.tile[slot][0], &sh.live[slot], sh.tile[free_slot][0], &sh.live[free_slot]);
        slot = slot + 1 == kRing<DT> ? 0 : slot + 1;
      }
    }
    const WaveTiles mine = {list, t0, t1, 1, kPageChunkTile};
    finish_rows<DT, CAP, BIAS>(p, table, head_off, q_row, sight, s.len, mine, st, f, lane);

    const int id = here(lane), last_h = id >> 5;
    const int last_row = row0 + kItemRows * wave + (id & 31);
    if (last_row < s.rows) {
      const int last_j = last_row / p.group;
      const int last_head = kh * p.group + (last_row - last_j * p.group);
      const int64_t last_query = s.start + last_j;
      const int64_t at = last_query * p.q_heads + last_head;
      const bool whole = p.splits == 1;
      const int64_t part_row = split * static_cast<int64_t>(p.n_tokens) * p.q_heads + at;
      char* dst = whole ? p.out + last_query * p.o_token + last_head * p.o_head
                        : reinterpret_cast<char*>(p.part_o + part_row * kHeadDim);
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int dim = 32 * d + 8 * a + 4 * last_h;
          const float z[4] = {st.o[d][4 * a], st.o[d][4 * a + 1], st.o[d][4 * a + 2], st.o[d][4 * a + 3]};
          if (whole)
            store4<DT>(dst + dim * ES, z);
          else
            store4<kF32>(dst + dim * 4, z);
        }
      if (last_h == 0) {
        if (!whole)
          p.part_ml[part_row] = make_float2(st.m, st.l);
        else if (p.lse)
          p.lse[at] = lse_of(st.m, st.l);
      }
    }
  }
}

template <int DT>
hipError_t launch_page_chunk(const PageAttendParams& p, dim3 grid, hipStream_t stream) {
  constexpr int kBytes = sizeof(PageChunkShared<DT>);
  auto* kernel = p.cap_log2 > 0.0f ? (p.slopes ? page_chunk_kernel<DT, true, true> : page_chunk_kernel<DT, true, false>)
                                   : (p.slopes ? page_chunk_kernel<DT, false, true> : page_chunk_kernel<DT, false, false>);
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, grid, dim3(kPageChunkThreads), kBytes, stream, p);
  return hipGetLastError();
}

}  // namespace hkv
