// Attention over records for many query rows per key head (prompts), included
// by one source per record format.
//
// A workgroup of 8 waves takes 256 rows of a key head (its query heads times
// the queries), 32 a wave, and walks the tokens in tiles of 64.  A tile's
// codes become fp16 once, in LDS, for all 8 waves:
//   keys    [64 tokens][128 dims], dims in the order of int4_run
//   values  [128 dims][64 tokens], the 8 tokens of an operand side by side
// both in 16-byte chunks whose place is XORed with the row, so that 8 lanes
// that read 8 rows, or write 8 chunks, meet different banks.
//
// The matrix instruction is 32x32x16 fp16, fp32 sums, keys and values its
// first operand, so that a lane (q, h) = (lane % 32, lane / 32) holds the
// scores of one row, tokens 8a + 4h + b of 32 in register 4a + b, which are
// the weights it has to supply to the second product: no exchange of lanes.
//
// Softmax as in attend_rows.h: a reference m per row that moves only when a
// tile's weights would leave fp16, weights below its normal numbers in passes
// of their own.  Here exp2 gives 2^14 times the weight, and the rows of a
// workgroup share one power of two (per row only where the rows' sizes differ
// by more than 2^14), so that scale, power and reference take one fused step.
//
// Waves 0..3 bring the tiles to come after their work on a tile, waves 4..7, on
// the same SIMDs, before it.  2,048 queries of 32 heads behind 16,384 tokens
// (8 key heads, INT4) take 0.96 to 1.1 ms, 470 to 540 TFLOP/s of the 1,280
// that a large library product reaches here (FP8 0.94; fp16 1.16 and fp32 2.0,
// with two parts; moved keys 1.5).  Of a tile's 7,200 clocks a wave
// spends 2 x 600 on scores, 2 x 1,000 on weights, 2 x 600 on the output, 1,100
// on bringing; two waves per SIMD overlap little of that, and a third does not
// fit the registers.  Products and weights interleaved in one instruction
// stream (1.28 ms) and waves half a tile apart (1.57 ms) spilled and were
// slower.
//
// Four tiles are under way at once: table entries, token offsets, codes,
// operands.
#pragma once

#include "attend_rows.h"

namespace hkv {

// A copy of x that the compiler takes for a new value: what is computed from
// it stays where it stands instead of holding registers across the loop.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kPromptTile = 64;

template <int DT, int QP>
struct PromptShared {
  char keys[2][kPromptTile * 256];
  char values[2][kHeadDim * 128];
  float ks[2][kPromptTile];            // token order: u, h, a, b of 32 u + 8 a + 4 h + b
  float vs[2][kPromptTile];
  int64_t vec[2][kPromptTile];         // byte offsets of the tokens' keys
  int64_t scale[2][kPromptTile];       // and of their key scales
  uint64_t live[4];                    // tokens of the tile that exist
  int32_t delta[4][kPromptTile];
  float top[kPromptWaves][2];          // largest and least row maximum of each wave
  float2 turn[QP > 1 ? kPromptWaves : 1][kHeadDim / 2];
  h8 low[QP > 1 ? kPromptWaves : 1][8][kWave];     // second parts of the queries: registers are few
};

template <int FMT, int DT, int QP>
// (two waves per SIMD, no more: the registers are for loads in flight)
__global__ __launch_bounds__(kPromptThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void attend_prompt_kernel(AttendParams p) {
  constexpr int CB = FMT == kFP8 ? kHeadDim : kHeadDim / 2;
  constexpr int W = CB / 64;
  constexpr int ES = ElemSize<DT>::value;
  constexpr int PP = DT == kBF16 ? 1 : 2;
  constexpr float kSmall = DT == kF32 ? 0x1p-3f : 0x1p-14f;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  PromptShared<DT, QP>& sh = *reinterpret_cast<PromptShared<DT, QP>*>(lds);
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int q32 = lane & 31, h = lane >> 5;

  const int kh = blockIdx.x % p.n_heads;
  const int rest = blockIdx.x / p.n_heads;
  const int split = rest % p.splits;
  const int r = blockIdx.y;
  const Span s = span_of(p, r);
  const int row_tiles = (s.rows + kPromptRows - 1) / kPromptRows;
  const int step = gridDim.x / (p.n_heads * p.splits);
  const int64_t v_off = static_cast<int64_t>(p.vecs) * CB;
  const int32_t* table = p.table + r * p.table_stride;
  const int32_t* moves = p.delta ? p.delta + r * p.table_stride : nullptr;

  // Later rows see more: they come first.
  for (int back = rest / p.splits; back < row_tiles; back += step) {
    const int row0 = (row_tiles - 1 - back) * kPromptRows;
    const int row = row0 + 32 * wave + q32;
    const int clamped = min(row, s.rows - 1);
    const int j = clamped / p.group;
    const int query = s.start + j;
    const int head = kh * p.group + (clamped - j * p.group);
    const char* q_row = p.q + query * p.q_token + head * p.q_head;
    const int sees = max(p.causal ? s.len - s.n_q + j + 1 : s.len, 0);
    // of the wave's rows: the fewest and the most tokens; of the workgroup's: the most
    const int wave_row = row0 + 32 * wave;
    const int j_first = min(wave_row, s.rows - 1) / p.group;
    const int j_last = min(wave_row + 31, s.rows - 1) / p.group;
    const int sees_least = p.causal ? s.len - s.n_q + j_first + 1 : s.len;
    const int sees_most = max(p.causal ? s.len - s.n_q + j_last + 1 : s.len, 0);
    const int j_end = (min(row0 + kPromptRows, s.rows) - 1) / p.group;
    const int sees_all = max(p.causal ? s.len - s.n_q + j_end + 1 : s.len, 0);
    const int tiles = sees_all / kPromptTile + (sees_all % kPromptTile != 0);
    const int per = (tiles + p.splits - 1) / p.splits;
    const int t0 = min(split * per, tiles);
    const int t1 = min(t0 + per, tiles);

    // Powers of two of the queries: the workgroup's, or each row's own.
    float top = 0.0f;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      float x[8];
      load8<DT>(q_row + (16 * kk + 8 * h) * ES, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
    }
    top = fmaxf(top, __shfl_xor(top, 32));
    // (A row that is not finite counts for neither: it has a power of its own.)
    const bool finite = top < INFINITY;
    float most = finite ? top : 0.0f, least = finite && top > 0.0f ? top : INFINITY;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      most = fmaxf(most, __shfl_xor(most, off));
      least = fminf(least, __shfl_xor(least, off));
    }
    __syncthreads();                     // the last rows' LDS is free
    if (lane == 0) {
      sh.top[wave][0] = most;
      sh.top[wave][1] = least;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPromptWaves; ++w) {
      most = fmaxf(most, sh.top[w][0]);
      least = fminf(least, sh.top[w][1]);
    }
    auto power = [](float t) {
      return t > 0.0f && t < INFINITY ? max(__builtin_amdgcn_frexp_expf(t) - 14, -100) : 0;
    };
    const int e_all = __builtin_amdgcn_readfirstlane(power(most));
    const bool uneven = __any(!finite) ||
                        __builtin_amdgcn_readfirstlane(least < INFINITY && power(least) < e_all - 14);
    const int e_row = uneven ? power(top) : e_all;
    const float even_out = __builtin_ldexpf(1.0f, e_row - e_all);
    const float ks_scale = p.scale_log2 * __builtin_ldexpf(1.0f, e_all);

    // Queries as operands: dims 16 kk + 8 h + (0 .. 7) in the order of the codes.
    h8 qf[8];
    h8* low = &sh.low[QP > 1 ? wave : 0][0][lane];
    auto to_operand = [&](const float (&x)[8], int kk) __attribute__((always_inline)) {
      h8 second;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        constexpr int kOrder[8] = {0, 4, 1, 5, 2, 6, 3, 7};
        const float v = __builtin_ldexpf(x[FMT == kINT4 ? kOrder[i] : i], -e_row);
        const _Float16 hi = static_cast<_Float16>(v);
        qf[kk][i] = hi;
        if constexpr (QP > 1) second[i] = static_cast<_Float16>(v - static_cast<float>(hi));
      }
      if constexpr (QP > 1) low[kk * kWave] = second;
    };
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      float x[8];
      load8<DT>(q_row + (16 * kk + 8 * h) * ES, x);
      to_operand(x, kk);
    }
    // the queries turned by -delta; a pair's dims lie in one lane
    auto turn_queries = [&](int delta) __attribute__((always_inline)) {
      float cc, ss;
      cos_sin(delta, p.theta[lane], &cc, &ss);
      float2* turn = sh.turn[QP > 1 ? wave : 0];
      wave_lds_fence();
      turn[lane] = make_float2(cc, -ss);
      wave_lds_fence();
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        float x[8], y[8];
        load8<DT>(q_row + (16 * kk + 8 * h) * ES, x);
        load8<DT>(q_row + (64 + 16 * kk + 8 * h) * ES, y);
        if (p.pairs == kInterleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a = turn[8 * kk + 4 * h + i], b = turn[32 + 8 * kk + 4 * h + i];
            turn_pair(x[2 * i], x[2 * i + 1], a.x, a.y);
            turn_pair(y[2 * i], y[2 * i + 1], b.x, b.y);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 a = turn[16 * kk + 8 * h + i];
            turn_pair(x[i], y[i], a.x, a.y);
          }
        }
        to_operand(x, kk);
        to_operand(y, kk + 4);
      }
    };
    int turned_by = 0;

    f32x16 o[4] = {};
    float m = kNoReference, l = 0.0f;
    bool far = false;                      // some row's reference is (kFar)

    // What this thread brings of a tile: 16 dims of a token's key, 8 dims of
    // two tokens' values (the pairs of a wave fill one chunk); waves 0 and 1 a
    // token's key or value scale per lane; wave 2 the tokens' places.
    auto k_token_of = [](int id) { return id >> 3; };
    auto v_token_of = [&](int id) {
      return 32 * (wave >> 2) + 16 * ((wave >> 1) & 1) + 4 * (wave & 1) + 2 * ((id >> 4) & 1) +
             8 * ((id >> 5) & 1);
    };
    u32x4 raw_k;                           // 8 (INT4) or 16 bytes (FP8)
    uint32_t raw_v[2][W];
    uint32_t raw_s = 0;
    int entry = 0, delta = 0;

    // Each step a wave works on tile t's scores, weights and output, and brings
    // tiles to come.  Waves 0..3 do the one first, waves 4..7, on the same
    // SIMDs, the other, so that the products of the ones meet the weights of
    // the others more often than their products.
    auto bring = [&](int t) __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);
      const int id = here(tid);
      const int k_token = k_token_of(id), k_part = id & 7, v_col = id & 15, v_token = v_token_of(id);
      // (tile t + 2's offsets: read first, they arrive behind the conversions)
      const int64_t k_off = sh.vec[t & 1][k_token];
      const int64_t v_offs[2] = {sh.vec[t & 1][v_token], sh.vec[t & 1][v_token + 1]};
      const int64_t s_off = sh.scale[t & 1][lane];
      const uint64_t live = sh.live[(t + 1) & 3];
      __builtin_amdgcn_sched_barrier(0);
      // Tile t + 1: codes to operands.
      if (t + 1 >= t0 && t + 1 < t1) {
        const int b = (t + 1) & 1;
        char* values = sh.values[b];
        char* krow = sh.keys[b] + k_token * 256;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          h8 x;
          if constexpr (FMT == kINT4)
            x = int4_run(raw_k[i]);
          else
            x = fp8_run(raw_k[2 * i], raw_k[2 * i + 1]);
          *reinterpret_cast<h8*>(krow + (((2 * k_part + i) ^ (k_token & 15)) << 4)) = x;
        }
        if (FMT == kFP8) {
          // codes of tokens that do not exist may be NaN
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (!((live >> (v_token + i)) & 1))
#pragma unroll
              for (int d = 0; d < W; ++d) raw_v[i][d] = 0;
        }
        h2 two[8];
        if constexpr (FMT == kINT4) {
          const uint32_t lo = __builtin_amdgcn_perm(raw_v[1][0], raw_v[0][0], 0x05040100u);
          const uint32_t hi = __builtin_amdgcn_perm(raw_v[1][0], raw_v[0][0], 0x07060302u);
          two[0] = nibble_low(lo);
          two[1] = nibble_high(lo);
          two[2] = nibble_low(lo >> 8);
          two[3] = nibble_high(lo >> 8);
          two[4] = nibble_low(hi);
          two[5] = nibble_high(hi);
          two[6] = nibble_low(hi >> 8);
          two[7] = nibble_high(hi >> 8);
        } else {
#pragma unroll
          for (int d = 0; d < W; ++d) {
            const uint32_t x = __builtin_amdgcn_perm(raw_v[1][d], raw_v[0][d], 0x05010400u);
            const uint32_t y = __builtin_amdgcn_perm(raw_v[1][d], raw_v[0][d], 0x07030602u);
            two[4 * d + 0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, false);
            two[4 * d + 1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, true);
            two[4 * d + 2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(y, 1.0f, false);
            two[4 * d + 3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(y, 1.0f, true);
          }
        }
        // tokens v_token, v_token + 1: chunk `wave`, halves 2 (lane / 16) and on
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int turned = i & 1 ? -(v_col >> 3) : v_col >> 3;       // i ^ (v_col >> 3) - i
          *reinterpret_cast<h2*>(values + (8 * v_col + turned) * 128 + 128 * i +
                                 ((wave ^ (v_col & 7)) << 4) + 4 * ((id >> 4) & 3)) = two[i];
        }
        if (wave < 2) {
          const float sc = (live >> lane) & 1 ? f16_bits_to_f32(raw_s) : 0.0f;
          const int at = 32 * (lane >> 5) + 16 * ((lane >> 2) & 1) + 4 * ((lane >> 3) & 3) + (lane & 3);
          if (wave == 0)
            sh.ks[b][at] = sc * ks_scale;
          else
            sh.vs[b][at] = sc;
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      // Tile t + 2: its codes and scales set out.
      if (t + 2 >= t0 && t + 2 < t1) {
        const uint8_t* ksrc = p.rec + k_off + 2 * W * 4 * k_part;
        if constexpr (FMT == kINT4) {
          const u32x2 x = *reinterpret_cast<const u32x2*>(ksrc);
          raw_k[0] = x[0];
          raw_k[1] = x[1];
        } else {
          raw_k = *reinterpret_cast<const u32x4*>(ksrc);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* vsrc = p.rec + v_offs[i] + v_off + 4 * W * v_col;
          if constexpr (W == 1) {
            raw_v[i][0] = *reinterpret_cast<const uint32_t*>(vsrc);
          } else {
            const u32x2 x = *reinterpret_cast<const u32x2*>(vsrc);
            raw_v[i][0] = x[0];
            raw_v[i][W - 1] = x[1];
          }
        }
        if (wave < 2)
          raw_s = *reinterpret_cast<const uint16_t*>(p.rec + s_off +
                                                     (wave == 0 ? 0 : 2 * static_cast<int64_t>(p.vecs)));
      }
      // Tiles t + 3 and t + 4: the tokens' offsets, and their table entries.
      // Tokens past the end stand for the last one, blocks outside the pool
      // for the first; neither is seen.
      if (wave == 2) {
        if (t + 3 >= t0 && t + 3 < t1) {
          const int tile = (t + 3) * kPromptTile;
          const int token = tile + min(lane, s.len - 1 - tile);
          const int block = static_cast<int>(
              (static_cast<uint64_t>(static_cast<uint32_t>(token)) * p.block_magic) >> p.block_shift);
          const bool known = static_cast<uint32_t>(entry) < static_cast<uint32_t>(p.n_blocks);
          const int64_t vec = static_cast<int64_t>(token - block * p.block_tokens) * p.n_heads + kh;
          const int64_t rec = (known ? entry : 0) * p.rec_block;
          sh.vec[(t + 3) & 1][lane] = rec + vec * CB;
          sh.scale[(t + 3) & 1][lane] = rec + 2 * v_off + 2 * vec;
          const uint64_t live = __ballot(known && lane < s.len - tile);
          if (lane == 0) sh.live[(t + 3) & 3] = live;
          if (QP > 1) sh.delta[(t + 3) & 3][lane] = delta;
        }
        if (t + 4 < t1) {
          const int tile = (t + 4) * kPromptTile;
          const int token = tile + min(lane, s.len - 1 - tile);
          const int block = static_cast<int>(
              (static_cast<uint64_t>(static_cast<uint32_t>(token)) * p.block_magic) >> p.block_shift);
          entry = table[block];
          if (QP > 1 && moves) delta = moves[block];
        }
      }
    };
    const bool early = wave >= kPromptWaves / 2;
    for (int t = t0 - 4; t < t1; ++t) {
      if (early) bring(t);
      {
        const int halves = t < t0 || t * kPromptTile >= sees_most ? 0 : 2;
#pragma unroll 1
        for (int u = 0; u < halves; ++u) {
          const uint32_t live = __builtin_amdgcn_readfirstlane(
              static_cast<uint32_t>(sh.live[t & 3] >> (32 * u)));
          const int first_token = t * kPromptTile + 32 * u;
          const bool part = live != ~0u || sees_least < 32 || first_token > sees_least - 32;
          f32x16 acc;
          // S^T = K Q^T
          const int k_at = here((32 * u + q32) * 256 + ((h ^ (q32 & 15)) << 4));
          auto scores = [&](f32x16& a) __attribute__((always_inline)) {
            a = f32x16{};
            // all reads first, so that the products wait once
            h8 kf[8];
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              kf[kk] = *reinterpret_cast<const h8*>(sh.keys[t & 1] + (k_at ^ (kk << 5)));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              if constexpr (QP > 1)
                a = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[kk], low[kk * kWave], a, 0, 0, 0);
              a = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[kk], qf[kk], a, 0, 0, 0);
            }
          };
          if (QP > 1 && moves) {
            // one pass per distance among the 32 tokens
            const int mine = sh.delta[t & 3][32 * u + q32];
            uint32_t left = live;
            bool first = true;
            do {
              const int d = __builtin_amdgcn_readlane(mine, left ? __builtin_ctz(left) : 0);
              const uint32_t same = static_cast<uint32_t>(__ballot(mine == d)) & left;
              if (left && d != turned_by) {
                turn_queries(d);
                turned_by = d;
              }
              f32x16 more;
              scores(more);
              const uint32_t take = first ? ~0u : same >> (4 * h);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                acc[i] = (take >> (8 * (i >> 2) + (i & 3))) & 1 ? more[i] : acc[i];
              left &= ~same;
              first = false;
            } while (left);
          } else {
            scores(acc);
          }
          if (uneven) {
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] *= even_out;
          }
          // dims of an operand's rows: 8 (row % 16) + row / 16 + 2 d, the lowest
          // bit turned over for dims 64 and on, which then take the other banks
          const int v_at = here((8 * (q32 & 15) + ((q32 >> 4) ^ ((q32 >> 3) & 1))) * 128);
          const int v_chunk[2] = {((4 * u + h) ^ (q32 & 7)) << 4, ((4 * u + 2 + h) ^ (q32 & 7)) << 4};
          auto value = [&](int d, int jj) __attribute__((always_inline)) {
            return *reinterpret_cast<const h8*>(sh.values[t & 1] + v_at + 256 * d + v_chunk[jj]);
          };
          // bit i: the row sees register i's token
          uint32_t vis = 0xFFFFu;
          if (part) {
            vis = 0;
            const uint32_t exist = live >> (4 * h);
            const int limit = sees - (first_token + 4 * h);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int in = 8 * (i >> 2) + (i & 3);
              vis |= ((exist >> in) & 1) && in < limit ? 1u << i : 0u;
            }
          }
          const float* ks = &sh.ks[t & 1][32 * u + 16 * h];
          const float* vs = &sh.vs[t & 1][32 * u + 16 * h];
          float w[16], sum, little;
          h8 pf[PP][2];
          auto parts = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const _Float16 hi = static_cast<_Float16>(w[i]);
              pf[0][i >> 3][i & 7] = hi;
              if constexpr (PP > 1)
                pf[1][i >> 3][i & 7] = static_cast<_Float16>(w[i] - static_cast<float>(hi));
            }
          };
          auto weights = [&]() __attribute__((always_inline)) {
            if (far) {
              // the reference came from rounded scores: so do the weights
#pragma clang fp contract(off)
              const float unit = fabsf(m) < kFar ? 14.0f : -3.0f;
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = (acc[i] * ks[i] - m) + unit;
            } else {
              const float shift = 14.0f - m;
#pragma unroll
              for (int a = 0; a < 4; ++a) {
                const f32x4 k4 = *reinterpret_cast<const f32x4*>(ks + 4 * a);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[4 * a + i] = __builtin_fmaf(acc[4 * a + i], k4[i], shift);
              }
            }
            if (part) {
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = (vis >> i) & 1 ? w[i] : -INFINITY;
            }
            sum = 0.0f;
#pragma unroll
            for (int a = 0; a < 4; ++a) {
              const f32x4 v4 = *reinterpret_cast<const f32x4*>(vs + 4 * a);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float e = __builtin_amdgcn_exp2f(w[4 * a + i]);
                sum += e;
                w[4 * a + i] = e * v4[i];
              }
            }
            if (part) {
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = (vis >> i) & 1 ? w[i] : 0.0f;
            }
          };
          weights();
          float big = 0.0f;
          little = INFINITY;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            big = fmaxf(big, fabsf(w[i]));
            little = fminf(little, fabsf(w[i]));
          }
          // Where a row's weights outgrow fp16, its reference moves: by a power of
          // two while they are finite, found anew where they are not (or where
          // the row does not see them all), or where weights of tokens without
          // values grow: 2^26 times 2^100 is the most that l then holds.
          const bool anew = __any(!(big < INFINITY) || sum > 0x1p100f);
          if (!anew && __any(big > 61440.0f)) {
            const float most_w = fmaxf(big, __shfl_xor(big, 32));
            const float up = most_w > 61440.0f ? rintf(__builtin_amdgcn_logf(most_w)) - 13.0f : 0.0f;
            const float keep = __builtin_ldexpf(1.0f, -static_cast<int>(up));
            m += up;
            l *= keep;
            sum *= keep;
            little *= keep;
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
              for (int i = 0; i < 16; ++i) o[d][i] *= keep;
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] *= keep;
          }
          if (anew) {
            float want = kNoReference;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float s2 = acc[i] * ks[i];
              const float lv = fminf(__builtin_amdgcn_logf(fabsf(vs[i])), 16.0f);
              const float x = fabsf(s2) < kFar ? fmaxf(s2 + lv, s2 - 80.0f) : s2;
              want = fmaxf(want, (vis >> i) & 1 ? x : kNoReference);
              if ((i & 7) == 7) __builtin_amdgcn_sched_barrier(0);    // few registers at a time
            }
            want = fmaxf(want, __shfl_xor(want, 32));
            const float m_new = fmaxf(m, rintf(want) + 1.0f);
            const float keep = m == m_new ? 1.0f : __builtin_amdgcn_exp2f(m - m_new);
            m = m_new;
            far = __any(fabsf(m) >= kFar && m > kNoReference);
            l *= keep;
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
              for (int i = 0; i < 16; ++i) o[d][i] *= keep;
            weights();
            little = 0.0f;
          }
          l += sum;
          parts();
          // O^T += V^T P^T
          __builtin_amdgcn_sched_barrier(0);
          {
            h8 vf[4][2];
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
              for (int jj = 0; jj < 2; ++jj) vf[d][jj] = value(d, jj);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int jj = 0; jj < 2; ++jj)
#pragma unroll
              for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int pp = PP - 1; pp >= 0; --pp)
                  o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[d][jj], pf[pp][jj], o[d], 0, 0, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
          if (__any(little < kSmall)) {
            // what rounding the weights to fp16 left out
            float unscale = 1.0f;
            for (int pass = 0; pass < 6; ++pass) {
              bool any = false;
#pragma unroll
              for (int i = 0; i < 16; ++i) any = any || (fabsf(w[i]) < kSmall && w[i] != 0.0f);
              if (!__any(any)) break;
              unscale *= 0x1p-28f;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float rem = w[i] - static_cast<float>(pf[0][i >> 3][i & 7]);
                if constexpr (PP > 1) rem -= static_cast<float>(pf[1][i >> 3][i & 7]);
                w[i] = fabsf(w[i]) < kSmall ? rem * 0x1p28f : 0.0f;
              }
              parts();
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                f32x16 add = {};
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                  const h8 vf = value(d, jj);
#pragma unroll
                  for (int pp = PP - 1; pp >= 0; --pp)
                    add = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, pf[pp][jj], add, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] = __builtin_fmaf(add[i], unscale, o[d][i]);
                __builtin_amdgcn_sched_barrier(0);
              }
            }
          }
        }
      }
      if (!early) bring(t);
      __syncthreads();
    }

    l += __shfl_xor(l, 32);
    const int last_row = row0 + 32 * wave + (here(tid) & 31);
    if (last_row < s.rows) {
      const int j = last_row / p.group;
      const int query = s.start + j;
      const int head = kh * p.group + (last_row - j * p.group);
      const int64_t at = static_cast<int64_t>(query) * p.q_heads + head;
      const bool whole = p.splits == 1;
      const bool empty = l == 0.0f;
      const float inv = !whole ? 1.0f : empty ? 0.0f : 1.0f / l;
      const int64_t part_row = split * static_cast<int64_t>(p.n_tokens) * p.q_heads + at;
      char* dst = whole ? p.out + query * p.o_token + head * p.o_head
                        : reinterpret_cast<char*>(p.part_o + part_row * kHeadDim);
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float y = o[i >> 1][8 * (i & 1) + 4 * a + b];
            x[i] = whole && empty ? 0.0f : y * inv;
          }
          const int dim = 8 * (8 * a + 4 * h + b);
          if (whole)
            store8<DT>(dst + dim * ES, x);
          else
            store8<kF32>(dst + dim * 4, x);
        }
      if (h == 0) {
        if (!whole)
          reinterpret_cast<float2*>(p.part_ml)[part_row] = make_float2(m, l * 0x1p-14f);
        else if (p.lse)
          p.lse[at] = log_sum(m - 14.0f, l);
      }
    }
  }
}

template <int FMT, int DT, int QP>
hipError_t launch_prompt_one(const AttendParams& p, dim3 grid, hipStream_t stream) {
  constexpr int kBytes = sizeof(PromptShared<DT, QP>);
  auto* kernel = attend_prompt_kernel<FMT, DT, QP>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, grid, dim3(kPromptThreads), kBytes, stream, p);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_prompt_format(const AttendParams& p, dim3 grid, hipStream_t stream) {
  switch (p.dtype) {
    case kF32:
      return launch_prompt_one<FMT, kF32, 2>(p, grid, stream);
    case kF16:
      return p.delta ? launch_prompt_one<FMT, kF16, 2>(p, grid, stream)
                     : launch_prompt_one<FMT, kF16, 1>(p, grid, stream);
    default:
      return p.delta ? launch_prompt_one<FMT, kBF16, 2>(p, grid, stream)
                     : launch_prompt_one<FMT, kBF16, 1>(p, grid, stream);
  }
}

}  // namespace hkv
