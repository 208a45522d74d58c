// Attention over records for few query rows per key head (decode, drafts),
// included by one source per record format.
//
// A key head's rows are its query heads times the request's queries; an item
// is up to 16 NT of them.  The matrix instruction is 16x16x32 fp16, fp32 sums:
//   scores  S^T = K Q^T    16 tokens x 16 rows, 4 steps of 32 dims
//   output  O^T = V^T P^T  16 dims x 16 rows, one step of 32 tokens
// so that the scores of a lane (one row, 8 tokens) are the very elements of
// P^T it has to supply: lane (c, g) = (lane % 16, lane / 16) takes tokens
// 8g .. 8g+7 of a tile of 32, rows 4g+i of the two score tiles standing for
// tokens 8g+i and 8g+4+i.  The order of a product's inner index is free, so
// codes are read as they lie: 16 (INT4) or 32 bytes (FP8) of a key per lane,
// 4 or 8 bytes of each of 8 values.
//
// Codes become fp16 exactly.  INT4: a nibble u = c ^ 8 put into the low
// mantissa bits of 1024 gives 1024 + c + 8 (or 1024 + 16 (c + 8) one nibble
// higher), and one packed fp16 step takes the offset off.  FP8: gfx950's
// conversion.  Queries are scaled by a power of two per row into fp16's range
// and split into two fp16 parts where one does not hold them (fp32 queries,
// queries turned by -delta); weights of fp32 queries likewise.
//
// Softmax: weights w = 2^14 exp2(s - m) v_scale enter their product as fp16, so
// m is a reference (a whole number) that keeps both w (fp16) and the sum's
// terms (fp32) finite.  It moves only when a tile would leave that range, to
// the tile's largest s + log2(v_scale) or largest s - 80: seldom after the
// first tile, which spares the rescaling of O and the reductions across lanes.
// Near the largest weight s - m is small, so its rounding is.  Weights below
// fp16's normal numbers, 2^-28 of the largest (2^-17 where two parts are to
// hold 22 bits), would lose their last bits, which shows where all heavier
// tokens have a code of 0: what rounding them left out follows in passes of
// its own, scaled up.
#pragma once

#include "attend_launch.h"
#include "rope_device.h"

namespace hkv {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Orders a wave's own LDS accesses for the compiler; the hardware keeps them
// in order.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ h2 nibble_low(uint32_t x) {
  const uint32_t y = (x & 0x000F000Fu) ^ 0x64086408u;
  const h2 off = {static_cast<_Float16>(1032.0f), static_cast<_Float16>(1032.0f)};
  return __builtin_bit_cast(h2, y) - off;
}
__device__ __forceinline__ h2 nibble_high(uint32_t x) {
  const uint32_t y = (x & 0x00F000F0u) ^ 0x64806480u;
  const h2 k = {static_cast<_Float16>(0.0625f), static_cast<_Float16>(0.0625f)};
  const h2 off = {static_cast<_Float16>(-72.0f), static_cast<_Float16>(-72.0f)};
  return __builtin_elementwise_fma(__builtin_bit_cast(h2, y), k, off);
}

// 8 INT4 codes of a dword as fp16, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ h8 int4_run(uint32_t x) {
  const uint32_t y = x >> 8;
  const h2 a = nibble_low(x), b = nibble_high(x), c = nibble_low(y), d = nibble_high(y);
  return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ h8 fp8_run(uint32_t lo, uint32_t hi) {
  const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  const h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  const h2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 8 dims x 8 tokens of V, one (INT4) or two (FP8) dwords per token, as 8
// operands: out[t] holds dim t of tokens 0 .. 7.
template <int FMT, int W>
__device__ __forceinline__ void transpose_run(const uint32_t (&v)[8][W], h8 (&out)[8]) {
  h2 part[8][4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (FMT == kINT4) {
      const uint32_t lo = __builtin_amdgcn_perm(v[2 * k + 1][0], v[2 * k][0], 0x05040100u);
      const uint32_t hi = __builtin_amdgcn_perm(v[2 * k + 1][0], v[2 * k][0], 0x07060302u);
      const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
      part[0][k] = nibble_low(lo);
      part[1][k] = nibble_high(lo);
      part[2][k] = nibble_low(lo8);
      part[3][k] = nibble_high(lo8);
      part[4][k] = nibble_low(hi);
      part[5][k] = nibble_high(hi);
      part[6][k] = nibble_low(hi8);
      part[7][k] = nibble_high(hi8);
    } else {
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const uint32_t x = __builtin_amdgcn_perm(v[2 * k + 1][d], v[2 * k][d], 0x05010400u);
        const uint32_t y = __builtin_amdgcn_perm(v[2 * k + 1][d], v[2 * k][d], 0x07030602u);
        part[4 * d + 0][k] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, false);
        part[4 * d + 1][k] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, true);
        part[4 * d + 2][k] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(y, 1.0f, false);
        part[4 * d + 3][k] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(y, 1.0f, true);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 8; ++t)
    out[t] = h8{part[t][0][0], part[t][0][1], part[t][1][0], part[t][1][1],
                part[t][2][0], part[t][2][1], part[t][3][0], part[t][3][1]};
}

__device__ __forceinline__ void load8_16bit(bool f16, const char* p, float (&x)[8]) {
  const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = a[j];
    x[2 * j] = f16 ? f16_bits_to_f32(w & 0xFFFFu) : bf16_bits_to_f32(w & 0xFFFFu);
    x[2 * j + 1] = f16 ? f16_bits_to_f32(w >> 16) : bf16_bits_to_f32(w >> 16);
  }
}
__device__ __forceinline__ void store8_any(int dtype, char* p, const float (&x)[8]) {
  if (dtype == kF32)
    store8<kF32>(p, x);
  else if (dtype == kF16)
    store8<kF16>(p, x);
  else
    store8<kBF16>(p, x);
}

struct Span {            // a request's queries and cached tokens
  int start, n_q, rows;  // rows: of a key head, of the queries that are computed
  int len;
};

__device__ __forceinline__ Span span_of(const AttendParams& p, int r) {
  Span s;
  s.start = p.q_start ? min(max(p.q_start[r], 0), p.n_tokens) : r;
  const int end = p.q_start ? min(max(p.q_start[r + 1], 0), p.n_tokens) : r + 1;
  s.n_q = max(end - s.start, 0);
  s.rows = min(s.n_q, p.max_queries) * p.group;
  s.len = min(max(p.kv_len[r], 0), p.max_len);
  return s;
}

__device__ __forceinline__ int tiles_of(const Span& s) {
  return max(s.len / kTileTokens + (s.len % kTileTokens != 0), 1);
}

constexpr float kNoReference = -3.0e38f;
constexpr float kLn2 = 0.69314718055994530942f;

constexpr float kWeightScale = 0x1p14f;

// log(2^m l), m a whole number; -infinity for l = 0.  Only the logarithm of
// l's significand is rounded before the last sum.
__device__ __forceinline__ float log_sum(float m, float l) {
  const int e = l > 0.0f && l < INFINITY ? __builtin_amdgcn_frexp_expf(l) : 0;
  return (__builtin_amdgcn_logf(__builtin_ldexpf(l, -e)) + (m + static_cast<float>(e))) * kLn2;
}

// State of a wave's rows: O^T by dim tile (lane (c, g): row c, dims
// 32 g + 8 i + t), the reference and the lane's part of the sum.
template <int NT>
struct RowState {
  f32x4 o[NT][8];
  float m[NT], l[NT];
};

template <int NT>
__device__ __forceinline__ void merge_rows(RowState<NT>& a, const f32x4* o, const float2* ml,
                                           int lane) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float2 b = ml[n * kWave + lane];
    const float m = fmaxf(a.m[n], b.x);
    const float fa = a.m[n] == m ? 1.0f : __builtin_amdgcn_exp2f(a.m[n] - m);
    const float fb = b.x == m ? 1.0f : __builtin_amdgcn_exp2f(b.x - m);
    a.m[n] = m;
    a.l[n] = a.l[n] * fa + b.y * fb;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const f32x4 x = o[(n * 8 + t) * kWave + lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) a.o[n][t][i] = a.o[n][t][i] * fa + x[i] * fb;
    }
  }
}

// QP, PP: fp16 parts of a query and of a weight.  TM: how block_tokens and
// the tile of 32 tokens fit: kWhole, a tile lies in one block; kEighths,
// runs of 8 tokens do; kAny.
enum TileMode { kWhole = 0, kEighths = 1, kAny = 2 };

template <int FMT, int NT, int QP, int PP, int TM>
__global__ __launch_bounds__(kRowsThreads, 2)
void attend_rows_kernel(AttendParams p) {
  constexpr int CB = FMT == kFP8 ? kHeadDim : kHeadDim / 2;
  constexpr int W = CB / 64;                  // dwords per 8 codes
  constexpr int kItemRows = 16 * NT;
  extern __shared__ char lds[];
  // per wave: scales of a tile (64 floats), token offsets (32 int64),
  // cosines and sines (64 float2); then the merge area; then the prefix
  struct WaveArea {
    float scale[2][kTileTokens];
    int64_t offset[kTileTokens];
    float2 turn[kHeadDim / 2];
  };
  static_assert(sizeof(WaveArea) == kWaveAreaBytes, "host LDS size");
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int c = lane & 15, g = lane >> 4;
  WaveArea& area = reinterpret_cast<WaveArea*>(lds)[wave];
  char* merge = lds + kRowsWaves * sizeof(WaveArea);
  f32x4* merge_o = reinterpret_cast<f32x4*>(merge);
  float2* merge_ml = reinterpret_cast<float2*>(merge + (kRowsWaves / 2) * NT * 8192);
  uint64_t* prefix = reinterpret_cast<uint64_t*>(merge + (kRowsWaves / 2) * NT * (8192 + 512));

  const int set = blockIdx.x % p.head_sets;
  const int range = blockIdx.x / p.head_sets;
  const int sub = wave % p.set_heads;
  const int phase = wave / p.set_heads;
  const int phases = kRowsWaves / p.set_heads;
  const int kh = set * p.set_heads + sub;
  const int64_t token_bytes = static_cast<int64_t>(p.n_heads) * CB;

  // The work: this workgroup's range of the tiles of all items, or (one
  // request per blockIdx.y) whole items.
  uint64_t at, end, per = 0, stride = 0;
  int r;
  if (p.ranges > 0) {
    const int R = p.n_requests;
    constexpr int kPer = kMaxFlatRequests / kRowsThreads;
    uint64_t own[kPer], sum = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int q = threadIdx.x * kPer + u;
      own[u] = 0;
      if (q < R) {
        const Span s = span_of(p, q);
        own[u] = static_cast<uint64_t>((s.rows + kItemRows - 1) / kItemRows) * tiles_of(s);
      }
      sum += own[u];
    }
    uint64_t run = sum;
    if (R > 1) {
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const uint64_t o = __shfl_up(run, off);
        if (lane >= off) run += o;
      }
    }
    uint64_t* wave_sum = reinterpret_cast<uint64_t*>(merge);
    if (lane == kWave - 1) wave_sum[wave] = run;
    __syncthreads();
    uint64_t before = run - sum;
    for (int w = 0; w < wave; ++w) before += wave_sum[w];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int q = threadIdx.x * kPer + u;
      if (q <= R) prefix[q] = before;
      before += own[u];
    }
    if (R == kMaxFlatRequests && threadIdx.x == kRowsThreads - 1) prefix[R] = before;
    __syncthreads();
    const uint64_t total = prefix[R];
    per = (total + p.ranges - 1) / p.ranges;
    if (per < static_cast<uint64_t>(p.min_tiles)) per = p.min_tiles;
    at = range * per;
    end = at + per < total ? at + per : total;
    if (p.prefix_out && blockIdx.x == 0) {
      for (int q = threadIdx.x; q <= R; q += kRowsThreads) p.prefix_out[q] = prefix[q];
      if (threadIdx.x == 0) p.prefix_out[R + 1] = per;
    }
    if (at >= end) return;
    int lo = 0, hi = R;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= at)
        lo = mid;
      else
        hi = mid;
    }
    r = lo;
  } else {
    r = blockIdx.y;
    const Span s = span_of(p, r);
    const uint64_t tiles = tiles_of(s);
    at = range * tiles;
    end = static_cast<uint64_t>((s.rows + kItemRows - 1) / kItemRows) * tiles;
    stride = static_cast<uint64_t>(gridDim.x / p.head_sets) * tiles;
    if (at >= end) return;
  }

  const uint64_t first_at = at;
  bool again = false;
  while (at < end) {
    if (again) __syncthreads();          // the merge area is free again
    again = true;
    if (p.ranges > 0)
      while (prefix[r + 1] <= at) ++r;   // requests without items
    const Span s = span_of(p, r);
    const int tiles = tiles_of(s);
    const uint64_t in_request = p.ranges > 0 ? at - prefix[r] : at;
    const int item = static_cast<int>(in_request / tiles);
    const int t0 = static_cast<int>(in_request - static_cast<uint64_t>(item) * tiles);
    int t1 = tiles;
    if (p.ranges > 0 && end - at < static_cast<uint64_t>(tiles - t0))
      t1 = t0 + static_cast<int>(end - at);
    const bool whole = t0 == 0 && t1 == tiles;
    const int row0 = item * kItemRows;

    // Rows of this lane, and what they see.
    const char* q_row[NT];
    int sees[NT], query[NT], head[NT];
    bool real[NT];
    int last = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = row0 + 16 * n + c;
      real[n] = row < s.rows;
      const int clamped = min(row, s.rows - 1);
      const int j = clamped / p.group;
      query[n] = s.start + j;
      head[n] = kh * p.group + (clamped - j * p.group);
      q_row[n] = p.q + query[n] * p.q_token + head[n] * p.q_head;
      sees[n] = max(p.causal ? s.len - s.n_q + j + 1 : s.len, 0);
    }
    const int j_first = row0 / p.group;
    const int j_last = (min(row0 + kItemRows, s.rows) - 1) / p.group;
    const int sees_least = p.causal ? s.len - s.n_q + j_first + 1 : s.len;
    const int sees_most = p.causal ? s.len - s.n_q + j_last + 1 : s.len;
    last = min(t1, max(sees_most, 0) / kTileTokens + (max(sees_most, 0) % kTileTokens != 0));

    const int32_t* table = p.table + r * p.table_stride;
    const int32_t* moves = p.delta ? p.delta + r * p.table_stride : nullptr;
    // Queries as operands: dims 32 g + 8 kk + (0 .. 7) in the order of the
    // codes, times 2^-e.  The row's exponent puts its largest magnitude below
    // 2^14, so a turned one stays below 2^15; fp16 queries that do not turn
    // are operands as they are.
    h8 qf[NT][QP][4];
    int e[NT];
    float grow[NT];                       // 2^e
    auto load_run = [&](const char* src, float (&x)[8]) __attribute__((always_inline)) {
      if constexpr (PP > 1)
        load8<kF32>(src, x);
      else
        load8_16bit(p.dtype == kF16, src, x);
    };
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float top = 0.0f;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        float x[8];
        load_run(q_row[n] + (32 * g + 8 * kk) * p.elem, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
      }
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      e[n] = 0;
      if (!(QP == 1 && p.dtype == kF16) && top > 0.0f && top < INFINITY)
        e[n] = max(__builtin_amdgcn_frexp_expf(top) - 14, -100);
      grow[n] = __builtin_ldexpf(1.0f, e[n]);
    }
    auto load_queries = [&](int delta) __attribute__((always_inline)) {
      if (QP > 1 && moves) {
        float cc, ss;
        cos_sin(delta, p.theta[lane], &cc, &ss);
        wave_lds_fence();
        area.turn[lane] = make_float2(cc, -ss);
        wave_lds_fence();
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          float x[8];
          load_run(q_row[n] + (32 * g + 8 * kk) * p.elem, x);
          if (QP > 1 && moves) {
            if (p.pairs == kInterleaved) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 t = area.turn[16 * g + 4 * kk + j];
                turn_pair(x[2 * j], x[2 * j + 1], t.x, t.y);
              }
            } else {
              float y[8];
              load_run(q_row[n] + (32 * (g ^ 2) + 8 * kk) * p.elem, y);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float2 t = area.turn[32 * (g & 1) + 8 * kk + j];
                float a = g < 2 ? x[j] : y[j], b = g < 2 ? y[j] : x[j];
                turn_pair(a, b, t.x, t.y);
                x[j] = g < 2 ? a : b;
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            constexpr int kOrder[8] = {0, 4, 1, 5, 2, 6, 3, 7};
            const float v = __builtin_ldexpf(x[FMT == kINT4 ? kOrder[j] : j], -e[n]);
            const _Float16 hi = static_cast<_Float16>(v);
            qf[n][0][kk][j] = hi;
            if constexpr (QP > 1) qf[n][1][kk][j] = static_cast<_Float16>(v - static_cast<float>(hi));
          }
        }
    };
    int turned_by = 0;
    bool loaded = false;
    if (QP == 1) load_queries(0);

    RowState<NT> st;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      st.m[n] = kNoReference;
      st.l[n] = 0.0f;
#pragma unroll
      for (int t = 0; t < 8; ++t) st.o[n][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // A tile on its way: the table entry and move of this lane's token
    // (8g+... of the tile: token lane % 32), then its codes and scales.
    struct Place {
      int block, entry, delta;
      int inside;                       // token within its block
    };
    auto place_of = [&](int t) __attribute__((always_inline)) {
      Place a;
      // tokens past the end stand for one that exists (kAny) or for a slot
      // of the last run of 8, which its block holds
      const int lim = s.len - 1 - t * kTileTokens;
      const int in_tile = lane & 31;
      const int token = t * kTileTokens + (TM == kWhole ? 0
                                           : TM == kEighths
                                               ? min(in_tile & ~7, lim & ~7) + (in_tile & 7)
                                               : min(in_tile, lim));
      a.block = static_cast<int>(
          (static_cast<uint64_t>(static_cast<uint32_t>(token)) * p.block_magic) >> p.block_shift);
      a.inside = token - a.block * p.block_tokens;
      a.entry = table[a.block];
      a.delta = QP > 1 && moves ? moves[a.block] : 0;
      return a;
    };
    struct Raw {
      u32x4 k[2][W];
      uint32_t v[8][W];
      uint32_t scale;
      uint32_t live;                    // tokens of the tile that exist
      int delta;
    };
    auto fetch = [&](int t, const Place& a) __attribute__((always_inline)) {
      Raw x;
      const bool ok = static_cast<uint32_t>(a.entry) < static_cast<uint32_t>(p.n_blocks) &&
                      (lane & 31) < s.len - t * kTileTokens;
      x.live = static_cast<uint32_t>(__ballot(ok));
      x.delta = a.delta;
      const int entry = static_cast<uint32_t>(a.entry) < static_cast<uint32_t>(p.n_blocks) ? a.entry : 0;
      const int64_t v_off = static_cast<int64_t>(p.vecs) * CB;
      if constexpr (TM == kWhole) {
        const uint8_t* rec = p.rec + __builtin_amdgcn_readfirstlane(entry) * p.rec_block;
        const int inside = __builtin_amdgcn_readfirstlane(a.inside);
        const uint8_t* kb = rec + inside * token_bytes + kh * CB;
        const uint32_t krow = (8 * (c >> 2) + (c & 3)) * static_cast<uint32_t>(token_bytes) + g * (CB / 4);
        const uint32_t vrow = 8 * g * static_cast<uint32_t>(token_bytes) + c * (CB / 16);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int w = 0; w < W; ++w)
            x.k[u][w] = *reinterpret_cast<const u32x4*>(kb + 4 * u * token_bytes + (krow + 16 * w));
        const uint8_t* vb = kb + v_off;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t* src = reinterpret_cast<const uint32_t*>(vb + k * token_bytes + vrow);
          if constexpr (W == 1) {
            x.v[k][0] = src[0];
          } else {
            const u32x2 y = *reinterpret_cast<const u32x2*>(src);
            x.v[k][0] = y[0];
            x.v[k][1] = y[1];
          }
        }
        const uint16_t* scales = reinterpret_cast<const uint16_t*>(rec + 2 * v_off) +
                                 (static_cast<int64_t>(inside) * p.n_heads + kh);
        x.scale = scales[(lane < 32 ? 0 : p.vecs) + (lane & 31) * p.n_heads];
      } else {
        const uint8_t* rec = p.rec + entry * p.rec_block;
        wave_lds_fence();
        if (lane < kTileTokens) area.offset[lane] = entry * p.rec_block + a.inside * token_bytes;
        wave_lds_fence();
        const uint8_t* kb = p.rec + kh * CB + g * (CB / 4);
        const uint8_t* vb = p.rec + kh * CB + c * (CB / 16) + v_off;
        const int64_t k0 = area.offset[8 * (c >> 2) + (TM == kAny ? c & 3 : 0)];
        const int64_t v0 = area.offset[8 * g];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint8_t* src;
          if constexpr (TM == kEighths)
            src = kb + k0 + ((c & 3) + 4 * u) * token_bytes;
          else
            src = kb + (u == 0 ? k0 : area.offset[8 * (c >> 2) + 4 + (c & 3)]);
#pragma unroll
          for (int w = 0; w < W; ++w) x.k[u][w] = *reinterpret_cast<const u32x4*>(src + 16 * w);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint8_t* at8 = vb + (TM == kEighths ? v0 + k * token_bytes : area.offset[8 * g + k]);
          if constexpr (W == 1) {
            x.v[k][0] = *reinterpret_cast<const uint32_t*>(at8);
          } else {
            const u32x2 y = *reinterpret_cast<const u32x2*>(at8);
            x.v[k][0] = y[0];
            x.v[k][1] = y[1];
          }
        }
        x.scale = reinterpret_cast<const uint16_t*>(rec + 2 * v_off)[
            (lane < 32 ? 0 : p.vecs) + a.inside * p.n_heads + kh];
      }
      return x;
    };

    auto scores = [&](const h8 (&kf)[2][4], f32x4 (&acc)[NT][2]) __attribute__((always_inline)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int qp = QP - 1; qp >= 0; --qp)
              a = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[u][kk], qf[n][qp][kk], a, 0, 0, 0);
          acc[n][u] = a;
        }
    };

    auto compute = [&](int t, Raw& x) __attribute__((always_inline)) {
      // wave-uniform
      const bool part = x.live != 0xFFFFFFFFu || sees_least < kTileTokens ||
                        t * kTileTokens > sees_least - kTileTokens;
      // scales through LDS: lane's token -> the 8 tokens of its group;
      // those of tokens that do not exist become 0
      const float sc = (x.live >> (lane & 31)) & 1 ? f16_bits_to_f32(x.scale) : 0.0f;
      wave_lds_fence();
      area.scale[lane >> 5][lane & 31] = sc * (lane < 32 ? p.scale_log2 : kWeightScale);
      wave_lds_fence();
      h8 kf[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if constexpr (FMT == kINT4) {
            kf[u][kk] = int4_run(x.k[u][0][kk]);
          } else {
            kf[u][kk] = fp8_run(x.k[u][kk >> 1][2 * (kk & 1)], x.k[u][kk >> 1][2 * (kk & 1) + 1]);
          }
        }
      f32x4 acc[NT][2];
      if constexpr (QP > 1) {
        // one pass per distance among the tile's tokens
        uint32_t left = x.live;
        bool first = true;
        do {
          const int lead = left ? __builtin_ctz(left) : 0;
          const int d = __builtin_amdgcn_readlane(x.delta, TM == kWhole ? 0 : lead);
          const uint32_t same = TM == kWhole ? left
                                             : static_cast<uint32_t>(__ballot(x.delta == d)) & left;
          if (!loaded || d != turned_by) load_queries(d);
          loaded = true;
          turned_by = d;
          f32x4 more[NT][2];
          scores(kf, more);
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool take = first || ((same >> (8 * g + 4 * u + i)) & 1);
#pragma unroll
              for (int n = 0; n < NT; ++n) acc[n][u][i] = take ? more[n][u][i] : acc[n][u][i];
            }
          left &= ~same;
          first = false;
        } while (left);
      } else {
        scores(kf, acc);
      }

      float ks[8], vs[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(&area.scale[0][8 * g + 4 * h]);
        const f32x4 b = *reinterpret_cast<const f32x4*>(&area.scale[1][8 * g + 4 * h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ks[4 * h + i] = a[i];
          vs[4 * h + i] = b[i];
        }
      }
      h8 pf[NT][PP];
      auto weights = [&](float (&w)[8], const float (&sv)[8], int n, float* sum) __attribute__((always_inline)) {
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sv[i], grow[n], -st.m[n]));
          total += e;
          w[i] = e * vs[i];
        }
        *sum = total;
      };
      auto split = [&](float y, int n, int i) __attribute__((always_inline)) {
        const _Float16 hi = static_cast<_Float16>(y);
        pf[n][0][i] = hi;
        if constexpr (PP > 1) pf[n][1][i] = static_cast<_Float16>(y - static_cast<float>(hi));
      };
      float sv[NT][8], w[NT][8], sum[NT];
      bool leave = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sv[n][i] = acc[n][i >> 2][i & 3] * ks[i];
        if (part) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const bool vis = ((x.live >> (8 * g + i)) & 1) && static_cast<uint32_t>(t * kTileTokens + 8 * g + i) <
                                                                     static_cast<uint32_t>(sees[n]);
            sv[n][i] = vis ? sv[n][i] : -INFINITY;
          }
        }
        weights(w[n], sv[n], n, &sum[n]);
        float top = fabsf(w[n][0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, fabsf(w[n][i]));
        leave = leave || top > 61440.0f || sum[n] > 0x1p96f;
      }
      if (__any(leave)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float want = kNoReference;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float s2 = sv[n][i] * grow[n];
            const float lv = fminf(__builtin_amdgcn_logf(fabsf(vs[i])) - 14.0f, 16.0f);
            want = fmaxf(want, fmaxf(s2 + lv, s2 - 80.0f));
          }
          want = fmaxf(want, __shfl_xor(want, 16));
          want = fmaxf(want, __shfl_xor(want, 32));
          const float m = fmaxf(st.m[n], rintf(want));
          const float keep = st.m[n] == m ? 1.0f : __builtin_amdgcn_exp2f(st.m[n] - m);
          st.m[n] = m;
          st.l[n] *= keep;
#pragma unroll
          for (int d = 0; d < 8; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.o[n][d][i] *= keep;
          weights(w[n], sv[n], n, &sum[n]);
        }
      }
      constexpr float kSmall = PP > 1 ? 0x1p-3f : 0x1p-14f;
      bool small = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        st.l[n] += sum[n];
        // a token that the row does not see weighs nothing whatever its scale
        if (part) {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[n][i] = sv[n][i] == -INFINITY ? 0.0f : w[n][i];
        }
        float least = fabsf(w[n][0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) least = fminf(least, fabsf(w[n][i]));
        small = small || least < kSmall;
#pragma unroll
        for (int i = 0; i < 8; ++i) split(w[n][i], n, i);
      }
      if (FMT == kFP8 && x.live != 0xFFFFFFFFu) {
        // codes of tokens that do not exist may be NaN
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int d = 0; d < W; ++d) x.v[k][d] = (x.live >> (8 * g + k)) & 1 ? x.v[k][d] : 0u;
      }
      h8 vf[8];
      transpose_run<FMT, W>(x.v, vf);
#pragma unroll
      for (int d = 0; d < 8; ++d)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int pp = PP - 1; pp >= 0; --pp)
            st.o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[d], pf[n][pp], st.o[n][d], 0, 0, 0);
      if (__any(small)) {
        float unscale = 1.0f;
        for (int pass = 0; pass < 5; ++pass) {
          bool any = false;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) any = any || (fabsf(w[n][i]) < kSmall && w[n][i] != 0.0f);
          if (!__any(any)) break;
          unscale *= 0x1p-28f;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float rest = w[n][i] - static_cast<float>(pf[n][0][i]);
              if constexpr (PP > 1) rest -= static_cast<float>(pf[n][1][i]);
              w[n][i] = fabsf(w[n][i]) < kSmall ? rest * 0x1p28f : 0.0f;
              split(w[n][i], n, i);
            }
#pragma unroll
          for (int d = 0; d < 8; ++d)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              f32x4 add = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
              for (int pp = PP - 1; pp >= 0; --pp)
                add = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[d], pf[n][pp], add, 0, 0, 0);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                st.o[n][d][i] = __builtin_fmaf(add[i], unscale, st.o[n][d][i]);
            }
        }
      }
    };

    int t = t0 + phase;
    if (t < last) {
      Place here = place_of(t);
      Place next = t + phases < last ? place_of(t + phases) : here;
      Raw raw = fetch(t, here);
      while (true) {
        const int t_next = t + phases;
        const bool more = t_next < last;
        Raw ahead = raw;
        if (more) {
          ahead = fetch(t_next, next);
          if (t_next + phases < last) next = place_of(t_next + phases);
        }
        compute(t, raw);
        if (!more) break;
        raw = ahead;
        t = t_next;
      }
    }

    // Phases join in halves, in a fixed order.
    for (int h = phases / 2; h > 0; h >>= 1) {
      __syncthreads();
      if (phase >= h && phase < 2 * h) {
        const int slot = (phase - h) * p.set_heads + sub;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          merge_ml[(slot * NT + n) * kWave + lane] = make_float2(st.m[n], st.l[n]);
#pragma unroll
          for (int d = 0; d < 8; ++d) merge_o[((slot * NT + n) * 8 + d) * kWave + lane] = st.o[n][d];
        }
      }
      __syncthreads();
      if (phase < h) {
        const int slot = phase * p.set_heads + sub;
        merge_rows<NT>(st, merge_o + slot * NT * 8 * kWave, merge_ml + slot * NT * kWave, lane);
      }
    }
    if (phase == 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float l = st.l[n] + __shfl_xor(st.l[n], 16);
        l += __shfl_xor(l, 32);
        if (!real[n]) continue;
        if (whole) {
          const bool empty = l == 0.0f;
          const float inv = empty ? 0.0f : 1.0f / (l * kWeightScale);
          char* dst = p.out + query[n] * p.o_token + head[n] * p.o_head;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x[8];
#pragma unroll
            for (int d = 0; d < 8; ++d) x[d] = empty ? 0.0f : st.o[n][d][i] * inv;
            store8_any(p.dtype, dst + (32 * g + 8 * i) * p.elem, x);
          }
          if (p.lse && g == 0)
            p.lse[static_cast<int64_t>(query[n]) * p.q_heads + head[n]] =
                log_sum(st.m[n], l);
        } else {
          const int64_t which = at == first_at ? 0 : 1;
          const int64_t row = (((static_cast<int64_t>(range) * 2 + which) * p.head_sets + set) *
                                   p.set_heads + sub) * p.part_rows + 16 * n + c;
          float* dst = p.part_o + row * kHeadDim;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x[8];
#pragma unroll
            for (int d = 0; d < 8; ++d) x[d] = st.o[n][d][i];
            store8<kF32>(reinterpret_cast<char*>(dst + 32 * g + 8 * i), x);
          }
          if (g == 0) reinterpret_cast<float2*>(p.part_ml)[row] = make_float2(st.m[n], l);
        }
      }
    }
    at += p.ranges > 0 ? static_cast<uint64_t>(t1 - t0) : stride;
  }
}

template <int FMT, int NT, int QP, int PP>
hipError_t launch_rows_tiles(const AttendParams& p, dim3 grid, size_t bytes, hipStream_t stream) {
  auto go = [&](auto* kernel) {
    // more than 64 KB of LDS has to be asked for
    if (bytes > 65536) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               hipFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(bytes));
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, grid, dim3(kRowsThreads), bytes, stream, p);
    return hipGetLastError();
  };
  if (p.block_tokens % kTileTokens == 0) return go(attend_rows_kernel<FMT, NT, QP, PP, kWhole>);
  if (p.block_tokens % 8 == 0) return go(attend_rows_kernel<FMT, NT, QP, PP, kEighths>);
  return go(attend_rows_kernel<FMT, NT, QP, PP, kAny>);
}

template <int FMT>
hipError_t launch_rows_format(const AttendParams& p, int nt, dim3 grid, size_t bytes,
                              hipStream_t stream) {
  if (p.dtype == kF32) return launch_rows_tiles<FMT, 1, 2, 2>(p, grid, bytes, stream);
  if (p.delta)
    return nt == 1 ? launch_rows_tiles<FMT, 1, 2, 1>(p, grid, bytes, stream)
                   : launch_rows_tiles<FMT, 2, 2, 1>(p, grid, bytes, stream);
  return nt == 1 ? launch_rows_tiles<FMT, 1, 1, 1>(p, grid, bytes, stream)
                 : launch_rows_tiles<FMT, 2, 1, 1>(p, grid, bytes, stream);
}

}  // namespace hkv
