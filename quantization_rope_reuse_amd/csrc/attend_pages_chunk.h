// Attention over pages for many query rows per key head (chunks of prompts,
// rows picked for recomputing).
//
// A workgroup of 4 waves takes 128 rows of a key head, 32 a wave, and walks the
// tokens that some of them see in tiles of 64 (fp32: 32), which each wave brings a
// quarter of into LDS and uses whole for its own rows; one barrier a tile, behind
// which the tile after next sets out.  Two workgroups fit a CU (80 KB of LDS, 256
// registers a lane; the 16-bit kernels spill none of them, those of fp32 three), so
// that one's barriers, first loads and last stores hide behind the other's products.
//
// Bound by issue: a wave's matrix instructions take 14 ns each, and of the vector
// work beside them (an exponential, a fused product, half a conversion, a sum and
// half a maximum a score) only about half hides behind them; a wave alone on its
// SIMD leaves the rest idle.  2,048 queries over 16,384 tokens (32 heads, 515
// GFLOP) take 528 to 546 us, 0.94 to 0.98 PFLOP/s, where the same products by the
// library's largest matrix product would take 410; 64 rows a wave with one wave a
// SIMD 780, 8 waves sharing a tile (half the loads into LDS, one workgroup a CU) 540
// where this took 524, and 179 for 158 with prompts of documents, whose items are
// short.
//
// Weights enter the second product rounded to the pages' type (2^-8 of each at most
// in bf16, 2^-11 in fp16): a second part of them would make half of the matrix work
// twice as long.  Against 64 bits a result's error is 1.4 times that of rounding it
// alone.
#pragma once

#include <type_traits>

#include "attend_pages.h"

namespace hkv {

template <int DT> constexpr int kChunkTile = DT == kF32 ? 32 : 64;     // tokens

// Step of a tile in 16-bit types: the products of the next one beside the weights
// of this one, then the output of this one beside the next's largest product
// (without cap and bias).  Matrix and vector instructions of one wave overlap
// only where they stand in turn, and reads of LDS only where they stand well
// ahead, so both are set out by hand and kept in place.
// bring(n), n = 0 .. 7: loads that set out in between.
template <int DT, bool MAX, class Bring>
__device__ __forceinline__ float tile_step(const f32x16 (&now)[2], RowsState& st, f32x16 (&next)[2], const char* next_keys,
                                           const char* values, const Queries<DT>& q, int lane, Bring bring) {
  constexpr int kSubBytes = kSub * Row<DT>::kBytes;
  const int id = here(lane);
  const int k_at = (id & 31) * Row<DT>::kBytes + (Row<DT>::key(id & 31, id >> 5) << 4);
  const int i16 = id & 15, v_token = 4 * (id >> 5) + (i16 >> 2);
  const int v_at = v_token * Row<DT>::kBytes + (Row<DT>::value(v_token, 2 * ((id >> 4) & 1) + ((i16 >> 1) & 1)) << 4) + 8 * (i16 & 1);
  auto key = [&](int u, int kk) __attribute__((always_inline)) {
    return *reinterpret_cast<const s8*>(next_keys + u * kSubBytes + (k_at ^ (kk << 5)));
  };
  auto value = [&](int u, int n) __attribute__((always_inline)) {      // n: 4 s + d
    const char* at = values + u * kSubBytes + (v_at ^ ((n & 3) << 6)) + 16 * (n >> 2) * Row<DT>::kBytes;
    const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS4)(at));
    const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS4)(at + 8 * Row<DT>::kBytes));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  // (each operand's registers take the one 8 products later)
  s8 a[8];
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) a[kk] = key(0, kk);
  __builtin_amdgcn_sched_barrier(0);
  // Weights two at a time, each stage of a pair one product behind the last, so
  // that none waits for the one before it.
  u32x4 w[2][2];                         // operands: 8 weights each
  float sum = 0.0f, x[2], e[2] = {};
  auto exponent = [&](int at) __attribute__((always_inline)) {
    return __builtin_fmaf(now[at >> 4][at & 15], st.scale, st.shift);
  };
  x[0] = exponent(0);
  x[1] = exponent(1);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    next[u] = f32x16{};
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const int pair = 8 * u + kk;
      next[u] = mma<DT>(a[kk], q.x[kk], next[u]);
      a[kk] = u == 0 ? key(1, kk) : value(0, kk);
      const float y0 = here(__builtin_amdgcn_exp2f(x[0])), y1 = here(__builtin_amdgcn_exp2f(x[1]));
      if (pair < 15) {
        x[0] = here(exponent(2 * pair + 2));
        x[1] = here(exponent(2 * pair + 3));
      }
      if (pair > 0) {
        sum = here(sum + e[0]);
        w[(pair - 1) >> 3][((pair - 1) >> 2) & 1][(pair - 1) & 3] = here(pack_two<DT>(e[0], e[1]));
        sum = here(sum + e[1]);
      }
      e[0] = y0;
      e[1] = y1;
      if (kk == 3 || kk == 6) bring(2 * u + (kk == 6));
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  w[1][1][3] = pack_two<DT>(e[0], e[1]);
  sum += e[0] + e[1];
  st.l += sum;
  float top = -INFINITY;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      st.o[n & 3] = mma<DT>(a[n], __builtin_bit_cast(s8, w[u][n >> 2]), st.o[n & 3]);
      if (u == 0) a[n] = value(1, n);
      if (n == 1 || n == 4) bring(4 + 2 * u + (n == 4));
      if (MAX) top = here(fmaxf(top, fmaxf(next[u][2 * n], next[u][2 * n + 1])));
      __builtin_amdgcn_sched_barrier(0);
    }
  return top;
}

template <int DT>
struct PageChunkShared {
  static constexpr int kTile = kChunkTile<DT>;
  char keys[2][kTile * Row<DT>::kBytes];     // (before the first tile: what the waves see)
  char values[3][kTile * Row<DT>::kBytes];
};

template <int DT, bool CAP, bool BIAS>
__global__ __launch_bounds__(kPageChunkThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void page_chunk_kernel(PageAttendParams p) {
  constexpr int ES = ElemSize<DT>::value;
  constexpr int kTile = kChunkTile<DT>;
  constexpr int N = kTile / kSub;
  using R = Row<DT>;
  constexpr int kRows = Group<DT>::kTokens;              // that a wave brings
  static_assert(kTile == kRows * kPageChunkWaves, "each wave brings a group");
  extern __shared__ __attribute__((aligned(16))) char lds[];
  PageChunkShared<DT>& sh = *reinterpret_cast<PageChunkShared<DT>*>(lds);
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int q32 = lane & 31, h = lane >> 5;

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
    int* bounds = reinterpret_cast<int*>(sh.keys);
    if (lane == 0) {
      bounds[3 * wave] = view.pre_most;
      bounds[3 * wave + 1] = view.lo_least;
      bounds[3 * wave + 2] = view.hi_most;
    }
    __syncthreads();
    int pre = 0, lo = INT32_MAX, hi = 0;
#pragma unroll
    for (int w = 0; w < kPageChunkWaves; ++w) {
      pre = max(pre, bounds[3 * w]);
      lo = min(lo, bounds[3 * w + 1]);
      hi = max(hi, bounds[3 * w + 2]);
    }
    __syncthreads();
    pre = __builtin_amdgcn_readfirstlane(pre);
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    const TileList list = tiles_of_view(pre, lo, hi, kTile);
    const int per = max((list.count + p.splits - 1) / p.splits, p.min_tiles);
    const int parts = max((list.count + per - 1) / per, 1);
    if (split >= parts) continue;
    const int t0 = split * per;
    const int t1 = min(t0 + per, list.count);

    RowsState st;
#pragma unroll
    for (int d = 0; d < 4; ++d) st.o[d] = f32x16{};
    st.m = kNoReference;
    st.l = 0.0f;
    st.far = false;

    // Each wave brings 16 tokens (fp32: 8) of a tile's keys and of its values.  The
    // table entries are read a tile ahead, each lane that of a token.
    const int group0 = kRows * wave;
    const typename Group<DT>::Lane key_lane(p, true, group0, lane), value_lane(p, false, group0, lane);
    int entry;
    auto find = [&](int t) __attribute__((always_inline)) {
      const int token = list.at(t) * kTile + (here(lane) & (kTile - 1));
      entry = table[block_of(p, min(token, s.len - 1))];
    };
    auto keys_of = [&](int t) __attribute__((always_inline)) { return sh.keys[(t - t0) & 1] + group0 * R::kBytes; };
    auto values_of = [&](int t) __attribute__((always_inline)) { return sh.values[(t - t0) % 3] + group0 * R::kBytes; };
    // Which of the tile's tokens exist.  Where all of the group do and lie in one
    // block, `rows` is their place, to be brought; else brings them, and it is -1.
    auto place = [&](int t, int64_t& rows) __attribute__((always_inline)) -> uint64_t {
      const int first = list.at(t) * kTile;
      const int token = first + (here(lane) & (kTile - 1));
      const bool known = token < s.len && static_cast<uint32_t>(entry) < static_cast<uint32_t>(p.num_pages);
      const uint64_t alive = __ballot(known);
      constexpr uint32_t kAll = (1u << kRows) - 1;
      if (p.grouped && (static_cast<uint32_t>(alive >> group0) & kAll) == kAll) {
        const int page = __builtin_amdgcn_readlane(entry, group0);
        const int at = first + group0;
        rows = page * p.page + (at - block_of(p, at) * p.block_tokens) * p.token + head_off;
      } else {
        rows = -1;
        const int in = group0 + (here(lane) & (kRows - 1));
        const int64_t at = Group<DT>::place(p, first + in, s.len, __shfl(entry, in), head_off);
        Group<DT>::bring_apart(p.k, at, true, group0, keys_of(t), here(lane));
        Group<DT>::bring_apart(p.v, at, false, group0, values_of(t), here(lane));
      }
      return alive;
    };
    auto bring_some = [&](int64_t rows, int n, char* keys, char* values) __attribute__((always_inline)) {
      if (n < 4)
        Group<DT>::bring_one(p, p.k + rows, key_lane, true, n, keys);
      else
        Group<DT>::bring_one(p, p.v + rows, value_lane, false, n - 4, values);
    };
    auto from_first = [&](int t) {
      return BIAS ? static_cast<float>(static_cast<double>(sight.pos) - (list.at(t) * kTile + 4 * h)) : 0.0f;
    };
    auto refer = [&](int t, f32x16 (&acc)[N], float top, uint64_t alive) __attribute__((always_inline)) {
      const int first = list.at(t) * kTile;
      const bool part = (alive << (64 - kTile)) != ~uint64_t{0} << (64 - kTile) || !view.all(first, kTile);
      refer_tile<DT, CAP, BIAS, N>(acc, top, st, f, part, part ? seen_of(sight, alive, first, h) : 0);
    };
    // Step t: the scores of tile t + 1 and the weights and output of tile t, whose
    // scores `now` holds; tile t + 2 sets out.  The areas do not overlap: reads of
    // some need not wait for loads of others.
    uint64_t live = 0;                     // of tile t + 1
    auto step = [&](int t, f32x16 (&now)[N], f32x16 (&next)[N], const char* __restrict__ next_keys,
                    const char* __restrict__ values, char* __restrict__ later_keys,
                    char* __restrict__ later_values) __attribute__((always_inline)) {
      int64_t rows = -1;
      uint64_t later_live = 0;
      if (t + 2 < t1) {
        later_live = place(t + 2, rows);
        find(min(t + 3, t1 - 1));
      }
      float top;
      if constexpr (DT == kF32) {
        if (rows >= 0) {
#pragma unroll
          for (int n = 0; n < 8; ++n) bring_some(rows, n, later_keys, later_values);
        }
#pragma unroll
        for (int u = 0; u < N; ++u) {
          next[u] = score_tile<DT>(next_keys + u * kSub * R::kBytes, q, lane);
          Weights<DT, 1> w;
          st.l += weigh_tile<DT, 1>(now[u], w, st);
          output_tile<DT, 1>(values + u * kSub * R::kBytes, w, st.o, lane);
        }
        top = scores_of<CAP, BIAS, N>(next, f, from_first(t + 1));
      } else {
        top = tile_step<DT, !CAP && !BIAS>(now, st, next, next_keys, values, q, lane, [&](int n) __attribute__((always_inline)) {
          if (rows >= 0) bring_some(rows, n, later_keys, later_values);
        });
        if (CAP || BIAS) top = scores_of<CAP, BIAS, N>(next, f, from_first(t + 1));
      }
      refer(t + 1, next, top, live);
      live = later_live;
    };
    if (t0 < t1) {
      f32x16 one[N], two[N];
      // Keys of tile t0 + n lie in slot n % 2, values in slot n % 3.
      find(t0);
      uint64_t first_live = 0;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if (t0 + n >= t1) break;
        int64_t rows;
        (n ? live : first_live) = place(t0 + n, rows);
        find(min(t0 + n + 1, t1 - 1));
        if (rows >= 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) bring_some(rows, i, keys_of(t0 + n), values_of(t0 + n));
        }
      }
      auto together = [&]() __attribute__((always_inline)) {
        // the loads of the last step, and everybody's reads of what the next ones replace
        wait_loads<0>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      };
      together();
#pragma unroll
      for (int u = 0; u < N; ++u) one[u] = score_tile<DT>(sh.keys[0] + u * kSub * R::kBytes, q, lane);
      refer(t0, one, scores_of<CAP, BIAS, N>(one, f, from_first(t0)), first_live);
      auto go = [&](int t, f32x16 (&now)[N], f32x16 (&next)[N]) __attribute__((always_inline)) {
        together();
        const int n = t - t0;
        step(t, now, next, sh.keys[(n + 1) & 1], sh.values[n % 3], keys_of(t + 2), values_of(t + 2));
      };
      int t = t0;
      for (; t + 2 < t1; t += 2) {
        go(t, one, two);
        go(t + 1, two, one);
      }
      if (t + 1 < t1) {
        go(t, one, two);
#pragma unroll
        for (int u = 0; u < N; ++u) one[u] = two[u];
      }
      together();
#pragma unroll
      for (int u = 0; u < N; ++u) {
        Weights<DT, 1> w;
        st.l += weigh_tile<DT, 1>(one[u], w, st);
        output_tile<DT, 1>(sh.values[(t1 - 1 - t0) % 3] + u * kSub * R::kBytes, w, st.o, lane);
      }
    }
    const WaveTiles mine = {list, t0, t1, 1, kTile};
    finish_rows<DT, 1, CAP, BIAS, N>(p, table, head_off, q_row, sight, s.len, mine, st, f, lane);

    const int id = here(lane), last_h = id >> 5;
    const int last_row = row0 + kItemRows * wave + (id & 31);
    if (last_row < s.rows) {
      const int last_j = last_row / p.group;
      const int last_head = kh * p.group + (last_row - last_j * p.group);
      const int64_t last_query = s.start + last_j;
      const int64_t at = last_query * p.q_heads + last_head;
      const bool whole = parts == 1;
      const int64_t part_row = split * static_cast<int64_t>(p.n_tokens) * p.q_heads + at;
      char* dst = whole ? p.out + last_query * p.o_token + last_head * p.o_head
                        : reinterpret_cast<char*>(p.part_o + part_row * kHeadDim);
      if (DT != kF32 && whole) {
        if constexpr (DT != kF32) {
          // Lanes q and q + 32 exchange halves: 8 dims in a row, 16 bytes, for each.
#pragma unroll
          for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int a = 0; a < 4; a += 2) {
              uint32_t z[4];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int at_a = 4 * a + 2 * i, at_b = at_a + 4;
                const auto both = __builtin_amdgcn_permlane32_swap(pack_two<DT>(st.o[d][at_a], st.o[d][at_a + 1]),
                                                                   pack_two<DT>(st.o[d][at_b], st.o[d][at_b + 1]), false, false);
                z[i] = both[0];
                z[2 + i] = both[1];
              }
              *reinterpret_cast<u32x4*>(dst + (32 * d + 8 * (a + last_h)) * ES) = u32x4{z[0], z[1], z[2], z[3]};
            }
        }
      } else {
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int a = 0; a < 4; ++a)
            store4<kF32>(dst + (32 * d + 8 * a + 4 * last_h) * 4,
                         {st.o[d][4 * a], st.o[d][4 * a + 1], st.o[d][4 * a + 2], st.o[d][4 * a + 3]});
      }
      if (last_h == 0) {
        if (p.splits > 1 && split == 0) p.part_n[at] = parts;
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
