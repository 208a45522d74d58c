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
// queries turned by -delta); weights likewise for fp32 and fp16 queries, whose
// results an 11-bit weight would show in.  (bf16 results have 8 bits: a second
// part would bring their error against 64 bits from 0.00167 to 0.00165 of their
// size, of moved keys from 0.00173 to 0.00171, and costs 1 to 4 % here, 15 % in
// the prompt kernel.)
//
// Softmax: weights w = 2^14 exp2(s - m) v_scale enter their product as fp16, so
// m is a reference (a whole number) that keeps both w (fp16) and the sum's
// terms (fp32) finite.  It moves only when a tile would leave that range, to a
// little above the tile's largest s + log2(v_scale) or the largest s - 80:
// seldom after the first tile, which spares the rescaling of O and the
// reductions across lanes.
// Near the largest weight s - m is small, so its rounding is.  Weights below
// fp16's normal numbers, 2^-28 of the largest (2^-17 where two parts are to
// hold 22 bits), would lose their last bits, which shows where all heavier
// tokens have a code of 0: what rounding them left out follows in passes of
// its own, scaled up.
//
// Work: the tiles of all items, dealt out evenly over about two workgroups of
// four waves per CU; a workgroup's waves take a range's tiles in turn (its
// phases) and join in LDS, and what reaches over several ranges is joined by
// attend_join_kernel.  Each wave has the next tile's codes under way while it
// works on one.
//
// What bounds it: 32 requests of up to 8,192 tokens (64 query heads over 8,
// INT4) take 43 to 47 us for 156 MB, 3.5 TB/s of the 6.2 that a large stream
// reaches, and 6 us to join.  A lone tile of two heads is some 450 vector instructions of 5 clocks (320 of them
// turn codes into fp16) beside 32 matrix instructions of 16; the waves' loops
// run at the rate of memory, but setting out (requests, queries, first codes:
// 13,000 of 90,000 clocks) and the join's waiting do not.  Wider layouts were
// slower: three or four waves per SIMD (72 to 77 us; spills), 1,024
// workgroups (59), 16 rows as two heads' rows apart (57).
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
// operands of which this makes four: out[t] holds dim 4 HALF + t of tokens
// 0 .. 7.
template <int FMT, int HALF, int W>
__device__ __forceinline__ void transpose_run(const uint32_t (&v)[8][W], h8 (&out)[4]) {
  h2 part[4][4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (FMT == kINT4) {
      const uint32_t x = __builtin_amdgcn_perm(v[2 * k + 1][0], v[2 * k][0],
                                               HALF == 0 ? 0x05040100u : 0x07060302u);
      const uint32_t y = x >> 8;
      part[0][k] = nibble_low(x);
      part[1][k] = nibble_high(x);
      part[2][k] = nibble_low(y);
      part[3][k] = nibble_high(y);
    } else {
      constexpr int d = W == 2 ? HALF : 0;
      const uint32_t x = __builtin_amdgcn_perm(v[2 * k + 1][d], v[2 * k][d], 0x05010400u);
      const uint32_t y = __builtin_amdgcn_perm(v[2 * k + 1][d], v[2 * k][d], 0x07030602u);
      part[0][k] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, false);
      part[1][k] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, true);
      part[2][k] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(y, 1.0f, false);
      part[3][k] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(y, 1.0f, true);
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t)
    out[t] = h8{part[t][0][0], part[t][0][1], part[t][1][0], part[t][1][1],
                part[t][2][0], part[t][2][1], part[t][3][0], part[t][3][1]};
}

__device__ __forceinline__ void store8_any(int dtype, char* p, const float (&x)[8]) {
  if (dtype == kF32)
    store8<kF32>(p, x);
  else if (dtype == kF16)
    store8<kF16>(p, x);
  else
    store8<kBF16>(p, x);
}

// A buffer from a wave-uniform address on: loads take a 32-bit offset per lane
// and one per wave, with no address arithmetic of their own.
__device__ __forceinline__ auto buffer_at(const uint8_t* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, 0xFFFFFFFFu, 0x00027000);
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

// From here on a reference has no bits for log2(v_scale) or for 14 beside a
// score, and moves by steps of its own: it takes the largest score alone, and
// weights are 2^-17 of the usual, which keeps them in fp16 whatever v_scale
// is (below 2^16).  Terms of one row that differ by those 2^17 are no further
// apart than scores of this size are exact.
constexpr float kFar = 0x1p23f;
constexpr float kFarBits = 17.0f;

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

// QP, PP: fp16 parts of a query (two for fp32 and for moved keys) and of a
// weight (two for fp32 and fp16).  TM: how block_tokens and the tile of 32
// tokens fit: kWhole, a tile lies in one block; kEighths, runs of 8 tokens do;
// kAny.
enum TileMode { kWhole = 0, kEighths = 1, kAny = 2 };

template <int FMT, int DT, int HP, int NT, int QP, int TM>
__global__ __launch_bounds__(kRowsThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void attend_rows_kernel(AttendParams p) {
  constexpr int CB = FMT == kFP8 ? kHeadDim : kHeadDim / 2;
  constexpr int W = CB / 64;                  // dwords per 8 codes
  constexpr int ES = ElemSize<DT>::value;
  constexpr int PP = DT == kBF16 ? 1 : 2;
  static_assert(HP == 1 || NT == 1, "two heads share one score tile");
  constexpr int kItemRows = 16 * NT / HP;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  // per wave: a WaveArea; then the merge area; then the prefix
  struct alignas(16) WaveArea {
    float scale[2][2][kTileTokens];      // K, V; head; token
    int64_t offset[kTileTokens];
    float2 turn[kHeadDim / 2];
  };
  static_assert(sizeof(WaveArea) == kWaveAreaBytes, "host LDS size");
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);   // uniform
  const int c = lane & 15, g = lane >> 4;
  WaveArea& area = reinterpret_cast<WaveArea*>(lds)[wave];
  char* merge = lds + kRowsWaves * sizeof(WaveArea);
  f32x4* merge_o = reinterpret_cast<f32x4*>(merge);
  float2* merge_ml = reinterpret_cast<float2*>(merge + (kRowsWaves / 2) * NT * 8192);
  uint32_t* prefix = reinterpret_cast<uint32_t*>(merge + (kRowsWaves / 2) * NT * (8192 + 512));

  const int set = blockIdx.x % p.head_sets;
  const int range = blockIdx.x / p.head_sets;
  const int sub = wave % p.set_heads;
  const int phase = wave / p.set_heads;
  const int phases = kRowsWaves / p.set_heads;
  const int kh0 = (set * p.set_heads + sub) * HP;      // the wave's first key head
  const int64_t token_bytes = static_cast<int64_t>(p.n_heads) * CB;

  // The work: this workgroup's range of the tiles of all items, or (one
  // request per blockIdx.y) whole items.
  uint32_t at = 0, end = 0;            // flat tiles
  int r = 0, item = range, items = 0;
  const int R = p.n_requests;
  const bool few = R <= kWave;         // a wave's lanes hold the requests' tiles
  uint32_t run = 0;                    // tiles up to and with this lane's request
  auto tiles_of_request = [&](int q) {
    const Span s = span_of(p, q);
    return static_cast<uint32_t>((s.rows + kItemRows - 1) / kItemRows) * tiles_of(s);
  };
  if (p.ranges > 0) {
    uint32_t total;
    if (few) {
      // every wave for itself, without LDS or a barrier
      run = lane < R ? tiles_of_request(lane) : 0;
      if (R > 1) {
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
          const uint32_t o = __shfl_up(run, off);
          if (lane >= off) run += o;
        }
      }
      total = __builtin_amdgcn_readlane(run, R - 1);
      if (lane >= R) run = total;
    } else {
      const int per_thread = (R + kRowsThreads - 1) / kRowsThreads;
      const int q0 = min(static_cast<int>(threadIdx.x) * per_thread, R);
      const int q1 = min(q0 + per_thread, R);
      uint32_t sum = 0;
      for (int q = q0; q < q1; ++q) sum += tiles_of_request(q);
      uint32_t upto = sum;
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const uint32_t o = __shfl_up(upto, off);
        if (lane >= off) upto += o;
      }
      uint32_t* wave_sum = reinterpret_cast<uint32_t*>(merge);
      if (lane == kWave - 1) wave_sum[wave] = upto;
      __syncthreads();
      uint32_t before = upto - sum;
      for (int w = 0; w < wave; ++w) before += wave_sum[w];
      for (int q = q0; q < q1; ++q) {
        prefix[q] = before;
        before += tiles_of_request(q);
      }
      if (threadIdx.x == kRowsThreads - 1) prefix[R] = before;   // its q1 is R
      __syncthreads();
      total = prefix[R];
    }
    const uint32_t per = max((total + p.ranges - 1) / p.ranges, static_cast<uint32_t>(p.min_tiles));
    at = min(range * per, total);       // range * per < total + per * ranges: below 2^32
    end = min(at + per, total);
    if (p.prefix_out && blockIdx.x == 0) {
      if (few) {
        if (wave == 0 && lane < R) p.prefix_out[lane + 1] = run;
        if (threadIdx.x == 0) p.prefix_out[0] = 0;
      } else {
        for (int q = threadIdx.x; q <= R; q += kRowsThreads) p.prefix_out[q] = prefix[q];
      }
      if (threadIdx.x == 0) p.prefix_out[R + 1] = per;
    }
    if (at >= end) return;
    if (!few) {
      int hi = R;
      while (hi - r > 1) {
        const int mid = (r + hi) >> 1;
        if (prefix[mid] <= at)
          r = mid;
        else
          hi = mid;
      }
    }
  } else {
    r = blockIdx.y;
    items = (span_of(p, r).rows + kItemRows - 1) / kItemRows;
  }

  const uint32_t first_at = at;
  bool again = false;
  while (p.ranges > 0 ? at < end : item < items) {
    if (again) __syncthreads();          // the merge area is free again
    again = true;
    uint32_t first = 0;                  // tiles before request r
    if (p.ranges > 0) {
      if (few) {
        r = __popcll(__ballot(run <= at));
        first = r > 0 ? __builtin_amdgcn_readlane(run, r - 1) : 0;
      } else {
        while (prefix[r + 1] <= at) ++r; // requests without items
        first = prefix[r];
      }
    }
    const Span s = span_of(p, r);
    const int tiles = tiles_of(s);
    int t0 = 0;
    if (p.ranges > 0) {
      item = (at - first) / static_cast<uint32_t>(tiles);
      t0 = at - first - item * tiles;
    }
    int t1 = tiles;
    if (p.ranges > 0 && end - at < static_cast<uint32_t>(tiles - t0))
      t1 = t0 + static_cast<int>(end - at);
    const bool whole = t0 == 0 && t1 == tiles;
    const int row0 = item * kItemRows;

    // Rows of this lane, and what they see.  (A division is some 30 instructions.)
    const bool one_query = s.rows <= p.group;
    const char* q_row[NT];
    int sees[NT], query[NT], head[NT];
    bool real[NT];
    int last = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = row0 + 16 * n + (HP == 2 ? c & 7 : c);
      real[n] = row < s.rows;
      const int clamped = min(row, s.rows - 1);
      const int j = one_query ? 0 : clamped / p.group;
      query[n] = s.start + j;
      head[n] = (HP == 2 ? kh0 + (c >> 3) : kh0) * p.group + (clamped - j * p.group);
      q_row[n] = p.q + query[n] * p.q_token + head[n] * p.q_head;
      sees[n] = max(p.causal ? s.len - s.n_q + j + 1 : s.len, 0);
    }
    const int j_first = one_query ? 0 : row0 / p.group;
    const int j_last = one_query ? 0 : (min(row0 + kItemRows, s.rows) - 1) / p.group;
    const int sees_least = p.causal ? s.len - s.n_q + j_first + 1 : s.len;
    const int sees_most = p.causal ? s.len - s.n_q + j_last + 1 : s.len;
    last = min(t1, max(sees_most, 0) / kTileTokens + (max(sees_most, 0) % kTileTokens != 0));

    // Queries as operands: dims 32 g + 8 kk + (0 .. 7) in the order of the
    // codes, times 2^-e.  The row's exponent puts its largest magnitude below
    // 2^14, so a turned one stays below 2^15; fp16 queries that do not turn
    // are operands as they are.
    h8 qf[NT][QP][4];
    int e[NT];
    float grow[NT];                       // 2^e
    const int32_t* table = p.table + r * p.table_stride;
    const int32_t* moves = p.delta ? p.delta + r * p.table_stride : nullptr;
    auto to_operand = [&](const float (&x)[8], int n, int kk) __attribute__((always_inline)) {
      h8 second;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        constexpr int kOrder[8] = {0, 4, 1, 5, 2, 6, 3, 7};
        const float v = __builtin_ldexpf(x[FMT == kINT4 ? kOrder[j] : j], -e[n]);
        const _Float16 hi = static_cast<_Float16>(v);
        qf[n][0][kk][j] = hi;
        if constexpr (QP > 1) second[j] = static_cast<_Float16>(v - static_cast<float>(hi));
      }
      if constexpr (QP > 1) qf[n][1][kk] = second;
    };
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float x[4][8], top = 0.0f;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) load8<DT>(q_row[n] + (32 * g + 8 * kk) * ES, x[kk]);
      e[n] = 0;
      if constexpr (!(QP == 1 && DT == kF16)) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[kk][j]));
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        if (top > 0.0f && top < INFINITY) e[n] = max(__builtin_amdgcn_frexp_expf(top) - 14, -100);
      }
      grow[n] = __builtin_ldexpf(1.0f, e[n]);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) to_operand(x[kk], n, kk);
    }
    // the queries turned by -delta
    auto turn_queries = [&](int delta) __attribute__((always_inline)) {
      float cc, ss;
      cos_sin(delta, p.theta[lane], &cc, &ss);
      wave_lds_fence();
      area.turn[lane] = make_float2(cc, -ss);
      wave_lds_fence();
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          float x[8], y[8];
          load8<DT>(q_row[n] + (32 * g + 8 * kk) * ES, x);
          if (p.pairs == kInterleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 t = area.turn[16 * g + 4 * kk + j];
              turn_pair(x[2 * j], x[2 * j + 1], t.x, t.y);
            }
          } else {
            load8<DT>(q_row[n] + (32 * (g ^ 2) + 8 * kk) * ES, y);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 t = area.turn[32 * (g & 1) + 8 * kk + j];
              float a = g < 2 ? x[j] : y[j], b = g < 2 ? y[j] : x[j];
              turn_pair(a, b, t.x, t.y);
              x[j] = g < 2 ? a : b;
            }
          }
          to_operand(x, n, kk);
        }
    };
    int turned_by = 0;

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
    struct Keys {
      u32x4 k[HP][2][W];
      uint32_t scale;
      uint32_t live;                    // tokens of the tile that exist
      int delta;
      const uint8_t* v;                 // this lane's values: first token (not kAny)
    };
    auto fetch_keys = [&](int t, const Place& a) __attribute__((always_inline)) {
      Keys x;
      const bool ok = static_cast<uint32_t>(a.entry) < static_cast<uint32_t>(p.n_blocks) &&
                      (lane & 31) < s.len - t * kTileTokens;
      x.live = static_cast<uint32_t>(__ballot(ok));
      x.delta = a.delta;
      const int entry = static_cast<uint32_t>(a.entry) < static_cast<uint32_t>(p.n_blocks) ? a.entry : 0;
      const int64_t v_off = static_cast<int64_t>(p.vecs) * CB;
      if constexpr (TM == kWhole) {
        const uint8_t* rec = p.rec + __builtin_amdgcn_readfirstlane(entry) * p.rec_block;
        const int inside = __builtin_amdgcn_readfirstlane(a.inside);
        const uint8_t* kb = rec + inside * token_bytes + kh0 * CB;
        x.v = kb + v_off;
        const auto keys = buffer_at(kb);
        const uint32_t krow = (8 * (c >> 2) + (c & 3)) * static_cast<uint32_t>(token_bytes) + g * (CB / 4);
#pragma unroll
        for (int h = 0; h < HP; ++h)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int w = 0; w < W; ++w)
              x.k[h][u][w] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                  keys, krow + h * CB + 16 * w, 4 * u * static_cast<uint32_t>(token_bytes), 0));
        const auto scales = buffer_at(rec + 2 * v_off + 2 * (static_cast<int64_t>(inside) * p.n_heads + kh0));
        const int at2 = 2 * ((lane < 32 ? 0 : p.vecs) + (lane & 31) * p.n_heads);
        // (two heads' scales lie side by side: one word)
        if constexpr (HP == 2)
          x.scale = __builtin_amdgcn_raw_buffer_load_b32(scales, at2, 0, 0);
        else
          x.scale = __builtin_amdgcn_raw_buffer_load_b16(scales, at2, 0, 0);
      } else {
        const uint8_t* rec = p.rec + entry * p.rec_block;
        wave_lds_fence();
        if (lane < kTileTokens) area.offset[lane] = entry * p.rec_block + a.inside * token_bytes;
        wave_lds_fence();
        const uint8_t* kb = p.rec + kh0 * CB + g * (CB / 4);
        const int64_t k0 = area.offset[8 * (c >> 2) + (TM == kAny ? c & 3 : 0)];
        x.v = p.rec + kh0 * CB + c * (CB / 16) + v_off + (TM == kEighths ? area.offset[8 * g] : 0);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint8_t* src;
          if constexpr (TM == kEighths)
            src = kb + k0 + ((c & 3) + 4 * u) * token_bytes;
          else
            src = kb + (u == 0 ? k0 : area.offset[8 * (c >> 2) + 4 + (c & 3)]);
#pragma unroll
          for (int h = 0; h < HP; ++h)
#pragma unroll
            for (int w = 0; w < W; ++w)
              x.k[h][u][w] = *reinterpret_cast<const u32x4*>(src + h * CB + 16 * w);
        }
        const uint16_t* scales = reinterpret_cast<const uint16_t*>(rec + 2 * v_off) +
                                 (lane < 32 ? 0 : p.vecs) + a.inside * p.n_heads + kh0;
        if constexpr (HP == 2)
          x.scale = *reinterpret_cast<const uint32_t*>(scales);
        else
          x.scale = *scales;
      }
      return x;
    };

    // (kAny: the tokens' offsets, in LDS since fetch_keys)
    auto fetch_values = [&](const Keys& x, uint32_t (&v)[HP][8][W]) __attribute__((always_inline)) {
      const uint32_t vrow = 8 * g * static_cast<uint32_t>(token_bytes) + c * (CB / 16);
#pragma unroll
      for (int h = 0; h < HP; ++h)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if constexpr (TM == kWhole) {
            const auto values = buffer_at(x.v);
            const uint32_t at8 = k * static_cast<uint32_t>(token_bytes);
            if constexpr (W == 1) {
              v[h][k][0] = __builtin_amdgcn_raw_buffer_load_b32(values, vrow + h * CB, at8, 0);
            } else {
              const u32x2 y = __builtin_bit_cast(
                  u32x2, __builtin_amdgcn_raw_buffer_load_b64(values, vrow + h * CB, at8, 0));
              v[h][k][0] = y[0];
              v[h][k][1] = y[1];
            }
          } else {
            const uint8_t* src = x.v + h * CB + (TM == kEighths ? k * token_bytes : area.offset[8 * g + k]);
            if constexpr (W == 1) {
              v[h][k][0] = *reinterpret_cast<const uint32_t*>(src);
            } else {
              const u32x2 y = *reinterpret_cast<const u32x2*>(src);
              v[h][k][0] = y[0];
              v[h][k][1] = y[1];
            }
          }
        }
    };

    // The scores of a tile.  Of two heads' a lane keeps its own head's: columns
    // 0..7 are rows of the first, 8..15 of the second.  The barriers keep the
    // operands of a step from being made before the last ones are used, which
    // would cost registers.
    auto scores = [&](const Keys& x, f32x4 (&acc)[NT][2]) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          h8 kf[4];
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if constexpr (FMT == kINT4)
              kf[kk] = int4_run(x.k[h][u][0][kk]);
            else
              kf[kk] = fp8_run(x.k[h][u][(kk >> 1) % W][2 * (kk & 1)],
                               x.k[h][u][(kk >> 1) % W][2 * (kk & 1) + 1]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
              for (int qp = QP - 1; qp >= 0; --qp) {
                a = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[kk], qf[n][qp][kk], a, 0, 0, 0);
              }
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[n][u][i] = h == 0 ? a[i] : (c >= 8 ? a[i] : acc[n][u][i]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
    };

    uint32_t v[HP][8][W];
    Keys x;
    Place next;
    int t = t0 + phase;
    if (t < last) {
      // Loads set out in the loop's order (keys, next place, values) here too:
      // the waits count loads in flight, by the worse of both ways in.
      x = fetch_keys(t, place_of(t));
      __builtin_amdgcn_sched_barrier(0);
      next = place_of(t + phases < last ? t + phases : t);
      __builtin_amdgcn_sched_barrier(0);
      fetch_values(x, v);
    }
    for (; t < last; t += phases) {
      // the tile after this one; the last one once more, to no use, keeps the
      // loads in flight countable
      const int after = t + phases < last ? t + phases : t;
      // wave-uniform
      const bool part = x.live != 0xFFFFFFFFu || sees_least < kTileTokens ||
                        t * kTileTokens > sees_least - kTileTokens;
      const uint32_t live = x.live;
      const uint32_t mine = live >> (8 * g);      // of this lane's 8 tokens
      const int delta = x.delta;
      // scales through LDS: lane's token -> the 8 tokens of its group;
      // those of tokens that do not exist become 0
      wave_lds_fence();
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        const float sc = (live >> (lane & 31)) & 1
                             ? f16_bits_to_f32(h == 0 ? x.scale & 0xFFFFu : x.scale >> 16) : 0.0f;
        area.scale[lane >> 5][h][lane & 31] = sc * (lane < 32 ? p.scale_log2 : kWeightScale);
      }
      wave_lds_fence();
      f32x4 acc[NT][2];
      if constexpr (QP > 1) {
        // one pass per distance among the tile's tokens
        uint32_t left = live;
        bool first = true;
        do {
          const int lead = left ? __builtin_ctz(left) : 0;
          const int d = __builtin_amdgcn_readlane(delta, TM == kWhole ? 0 : lead);
          const uint32_t same = TM == kWhole ? left
                                             : static_cast<uint32_t>(__ballot(delta == d)) & left;
          if (d != turned_by) turn_queries(d);
          turned_by = d;
          f32x4 more[NT][2];
          scores(x, more);
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool take = first || (((same >> (8 * g)) >> (4 * u + i)) & 1);
#pragma unroll
              for (int n = 0; n < NT; ++n) acc[n][u][i] = take ? more[n][u][i] : acc[n][u][i];
            }
          left &= ~same;
          first = false;
        } while (left);
      } else {
        scores(x, acc);
      }

      // the next tile's keys set out as soon as this one's registers are free,
      // its values once this tile's are used
      x = fetch_keys(after, next);
      __builtin_amdgcn_sched_barrier(0);
      next = place_of(after + phases < last ? after + phases : after);
      float ks[8], vs[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(&area.scale[0][HP == 2 ? c >> 3 : 0][8 * g + 4 * h]);
        const f32x4 b = *reinterpret_cast<const f32x4*>(&area.scale[1][HP == 2 ? c >> 3 : 0][8 * g + 4 * h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ks[4 * h + i] = a[i];
          vs[4 * h + i] = b[i];
        }
      }
      h8 pf[NT][PP];
      auto weights = [&](float (&w)[8], const float (&sv)[8], int n,
                         float* sum, float less) __attribute__((always_inline)) {
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sv[i], grow[n], -st.m[n]) - less);
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
      float big[NT];
      bool leave = false, anew = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sv[n][i] = acc[n][i >> 2][i & 3] * ks[i];
        if (part) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const bool vis = ((mine >> i) & 1) && static_cast<uint32_t>(t * kTileTokens + 8 * g + i) <
                                                      static_cast<uint32_t>(sees[n]);
            sv[n][i] = vis ? sv[n][i] : -INFINITY;
          }
        }
        weights(w[n], sv[n], n, &sum[n], 0.0f);
        // a token that the row does not see weighs nothing whatever its scale
        if (part) {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[n][i] = sv[n][i] == -INFINITY ? 0.0f : w[n][i];
        }
        big[n] = fabsf(w[n][0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) big[n] = fmaxf(big[n], fabsf(w[n][i]));
        leave = leave || big[n] > 61440.0f;
        anew = anew || !(big[n] < INFINITY) || sum[n] > 0x1p96f;
      }
      // Where a row's weights outgrow fp16, its reference moves: by a power of
      // two while they are finite, found anew where they are not.
      // (Of 32 rows always anew: both ways would cost the usual one registers.)
      anew = __any(NT == 1 ? anew : anew || leave);
      if (NT == 1 && !anew && __any(leave)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float most = fmaxf(big[n], __shfl_xor(big[n], 16));
          most = fmaxf(most, __shfl_xor(most, 32));
          const float up = most > 61440.0f ? rintf(__builtin_amdgcn_logf(most)) - 13.0f : 0.0f;
          const float keep = __builtin_ldexpf(1.0f, -static_cast<int>(up));
          st.m[n] += up;
          st.l[n] *= keep;
          sum[n] *= keep;
#pragma unroll
          for (int d = 0; d < 8; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.o[n][d][i] *= keep;
#pragma unroll
          for (int i = 0; i < 8; ++i) w[n][i] *= keep;
        }
      }
      if (anew) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float want = kNoReference;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float s2 = sv[n][i] * grow[n];
            const float lv = fminf(__builtin_amdgcn_logf(fabsf(vs[i])) - 14.0f, 16.0f);
            want = fmaxf(want, fabsf(s2) < kFar ? fmaxf(s2 + lv, s2 - 80.0f) : s2);
          }
          want = fmaxf(want, __shfl_xor(want, 16));
          want = fmaxf(want, __shfl_xor(want, 32));
          const float m = fmaxf(st.m[n], rintf(want) + 1.0f);
          const float keep = st.m[n] == m ? 1.0f : __builtin_amdgcn_exp2f(st.m[n] - m);
          st.m[n] = m;
          st.l[n] *= keep;
#pragma unroll
          for (int d = 0; d < 8; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.o[n][d][i] *= keep;
          weights(w[n], sv[n], n, &sum[n], fabsf(m) < kFar ? 0.0f : kFarBits);
          if (part) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[n][i] = sv[n][i] == -INFINITY ? 0.0f : w[n][i];
          }
        }
      }
      constexpr float kSmall = DT == kF32 ? 0x1p-3f : 0x1p-14f;
      bool small = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        st.l[n] += sum[n];
        float least = fabsf(w[n][0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) least = fminf(least, fabsf(w[n][i]));
        small = small || least < kSmall;
#pragma unroll
        for (int i = 0; i < 8; ++i) split(w[n][i], n, i);
      }
      if (FMT == kFP8 && live != 0xFFFFFFFFu) {
        // codes of tokens that do not exist may be NaN
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int h = 0; h < HP; ++h)
#pragma unroll
            for (int d = 0; d < W; ++d) v[h][k][d] = (mine >> k) & 1 ? v[h][k][d] : 0u;
      }
      // a head's values meet its own rows' weights, 0 in the other's columns
      auto own = [&](const h8& w8, int h) __attribute__((always_inline)) {
        if constexpr (HP == 1) return w8;
        const u32x4 y = __builtin_bit_cast(u32x4, w8);
        u32x4 z;
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = (c >= 8) == (h == 1) ? y[i] : 0u;
        return __builtin_bit_cast(h8, z);
      };
      // O^T += V^T P^T, four dim tiles at a time; or of weights
      // that were scaled up
      auto output = [&](float unscale, bool scaled) __attribute__((always_inline)) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int h = 0; h < HP; ++h) {
            h8 vf[4];
            if (half == 0)
              transpose_run<FMT, 0, W>(v[h], vf);
            else
              transpose_run<FMT, 1, W>(v[h], vf);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int pp = PP - 1; pp >= 0; --pp) {
                const h8 w8 = own(pf[n][pp], h);
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                  f32x4& o = st.o[n][4 * half + d];
                  if (!scaled) {
                    o = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[d], w8, o, 0, 0, 0);
                  } else {
                    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
                    const f32x4 add = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[d], w8, zero, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(add[i], unscale, o[i]);
                  }
                }
              }
            __builtin_amdgcn_sched_barrier(0);
          }
      };
      output(1.0f, false);
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
          output(unscale, true);
        }
      }
      fetch_values(x, v);
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
            store8<DT>(dst + (32 * g + 8 * i) * ES, x);
          }
          if (p.lse && g == 0)
            p.lse[static_cast<int64_t>(query[n]) * p.q_heads + head[n]] =
                log_sum(st.m[n], l);
        } else {
          const int64_t which = at == first_at ? 0 : 1;
          const int64_t row = ((static_cast<int64_t>(range) * 2 + which) * p.n_heads +
                               (HP == 2 ? kh0 + (c >> 3) : kh0)) * p.part_rows +
                              16 * n + (HP == 2 ? c & 7 : c);
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
    at += t1 - t0;
    if (p.ranges == 0) item += gridDim.x / p.head_sets;
  }
}

template <int FMT, int DT, int HP, int NT, int QP>
hipError_t launch_rows_tiles(const AttendParams& p, dim3 grid, size_t bytes, hipStream_t stream) {
  auto go = [&](auto* kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kRowsThreads), bytes, stream, p);
    return hipGetLastError();
  };
  if (p.block_tokens % kTileTokens == 0) return go(attend_rows_kernel<FMT, DT, HP, NT, QP, kWhole>);
  if (p.block_tokens % 8 == 0) return go(attend_rows_kernel<FMT, DT, HP, NT, QP, kEighths>);
  return go(attend_rows_kernel<FMT, DT, HP, NT, QP, kAny>);
}

// hp, nt: two heads per score tile, or 16 nt rows of one.
template <int FMT, int DT>
hipError_t launch_rows_dtype(const AttendParams& p, int hp, int nt, dim3 grid, size_t bytes,
                             hipStream_t stream) {
  // two parts per query: 32 rows of them leave the registers, and 16 rows
  // twice over are faster (54 against 145 us for drafts of five tokens of 16
  // requests over FP8 records)
  auto two_parts = [&] {
    return hp == 2 ? launch_rows_tiles<FMT, DT, 2, 1, 2>(p, grid, bytes, stream)
                   : launch_rows_tiles<FMT, DT, 1, 1, 2>(p, grid, bytes, stream);
  };
  if constexpr (DT == kF32) {
    return two_parts();
  } else {
    if (p.delta) return two_parts();
    if (hp == 2) return launch_rows_tiles<FMT, DT, 2, 1, 1>(p, grid, bytes, stream);
    return nt == 1 ? launch_rows_tiles<FMT, DT, 1, 1, 1>(p, grid, bytes, stream)
                   : launch_rows_tiles<FMT, DT, 1, 2, 1>(p, grid, bytes, stream);
  }
}

template <int FMT>
hipError_t launch_rows_format(const AttendParams& p, int hp, int nt, dim3 grid, size_t bytes,
                              hipStream_t stream) {
  switch (p.dtype) {
    case kF32: return launch_rows_dtype<FMT, kF32>(p, hp, nt, grid, bytes, stream);
    case kF16: return launch_rows_dtype<FMT, kF16>(p, hp, nt, grid, bytes, stream);
    default: return launch_rows_dtype<FMT, kBF16>(p, hp, nt, grid, bytes, stream);
  }
}

}  // namespace hkv
