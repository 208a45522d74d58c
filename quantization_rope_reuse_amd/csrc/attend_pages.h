// Attention over pages, included by one source per element type.
//
// A key head's rows are its query heads times the request's queries.  A wave
// takes 32 of them and walks the cached tokens in subtiles of 32 with the
// matrix instruction 32x32 (16 inner steps in 16-bit types, 2 in fp32), fp32
// sums, keys and values its first operand:
//   scores  S^T = K Q^T    32 tokens x 32 rows
//   output  O^T = V^T P^T  4 times 32 dims x 32 rows
// so that a lane (q, h) = (lane % 32, lane / 32) holds scores of one row,
// tokens 8a + 4h + b in register 4a + b, which are the weights it has to supply
// to the second product (whose inner order is free): no exchange of lanes.
//
// Tiles lie in LDS as they lie in the pages, a token's 128 dims a row; tokens
// that do not exist are read from a place of zeros.  Rows are cut in chunks of
// 16 bytes whose place is XORed with the token, so that lanes reading the same
// chunk of several tokens meet different banks.  Values reach the operand,
// which wants several tokens of one dim, through gfx950's transposing LDS read.
//
// Softmax: weights w = exp2(s - m + kOff) with a whole reference m per row that
// moves only when a tile's scores exceed it by kSlack, which spares most tiles
// the rescaling of O and the reduction across lanes.  16-bit floats keep their
// weights in the type's normal numbers down to 2^-(14 + kOff) of the reference
// (fp16); bf16's and fp32's range needs no offset.
//
// A masked token's weight is 0, but 0 times an infinite value is not: where a
// row's sum is finite and its output is not, the wave makes its output again with
// such values apart (output_again).
#pragma once

#include <type_traits>

#include "attend_pages_launch.h"
#include "attend_pages_tiles.h"
#include "hkv_device.h"

namespace hkv {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef short s8 __attribute__((ext_vector_type(8)));

constexpr int kSub = 32;                   // tokens of a subtile
constexpr float kNoReference = -3.4028234663852886e38f;     // the least: no score lies below it
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kFar = 0x1p16f;            // references from here on: scores are rounded before m is taken off

// Where tokens that do not exist are read.
__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0, 0, 0, 0};

template <int DT> struct PageTraits;
template <> struct PageTraits<kBF16> {
  static constexpr float kOff = 0.0f, kSlack = 8.0f;
};
template <> struct PageTraits<kF16> {
  static constexpr float kOff = 12.0f, kSlack = 3.0f;
};
template <> struct PageTraits<kF32> {
  static constexpr float kOff = 0.0f, kSlack = 8.0f;
};

// Geometry of a token's row in LDS.
template <int DT>
struct Row {
  static constexpr int ES = ElemSize<DT>::value;
  static constexpr int kBytes = kHeadDim * ES;
  static constexpr int kChunks = kBytes / 16;       // lanes that bring one row
  static constexpr int kPerWave = kWave / kChunks;  // rows of a wave's load
  static __device__ __forceinline__ int key(int token, int chunk) { return chunk ^ (token & 15); }
  static __device__ __forceinline__ int value(int token, int chunk) {
    return DT == kF32 ? chunk ^ (2 * (token & 4)) : chunk ^ (4 * (token & 3));
  }
};

struct PageSpan {        // a request's queries and cached tokens
  int start, n_q, rows;  // rows: of a key head, of the queries that are computed
  int len, pre;          // pre: tokens of the prefix
};

// (An array that is not there is read elsewhere, so that the loads need not
// wait for each other.)
__device__ __forceinline__ PageSpan page_span(const PageAttendParams& p, int r) {
  const int32_t* bounds = p.q_start ? p.q_start + r : p.kv_len;
  const int32_t* prefix = p.prefix ? p.prefix : p.kv_len;
  const int from = bounds[0], to = p.q_start ? bounds[1] : 0, len = p.kv_len[r], pre = prefix[r];
  PageSpan s;
  s.start = p.q_start ? min(max(from, 0), p.n_tokens) : r;
  const int end = p.q_start ? min(max(to, 0), p.n_tokens) : r + 1;
  s.n_q = max(end - s.start, 0);
  s.rows = min(s.n_q, p.max_queries) * p.group;
  s.len = min(max(len, 0), p.max_len);
  s.pre = p.prefix ? min(max(pre, 0), s.len) : 0;
  return s;
}

struct Sight {           // tokens [0, pre) and [lo, hi), hi >= lo
  int pre, lo, hi;
  int pos;
};

// What row j of a request sees.
__device__ __forceinline__ Sight sight_of(const PageAttendParams& p, const PageSpan& s, int j) {
  Sight v;
  const int query = s.start + j;
  v.pos = p.positions ? p.positions[query] : s.len - s.n_q + j;
  if (p.positions && v.pos < 0) return {0, 0, 0, v.pos};
  const int at = max(v.pos, -1);
  v.pre = s.pre;
  v.hi = p.causal ? min(at, s.len - 1) + 1 : s.len;
  v.lo = p.begin ? max(p.begin[query], 0) : 0;
  if (p.window > 0) v.lo = max(v.lo, at - p.window + 1);
  v.lo = min(v.lo, v.hi);
  return v;
}

__device__ __forceinline__ int wave_min(int x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x = min(x, __shfl_xor(x, off));
  return __builtin_amdgcn_readfirstlane(x);
}
__device__ __forceinline__ int wave_max(int x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x = max(x, __shfl_xor(x, off));
  return __builtin_amdgcn_readfirstlane(x);
}

// What a set of rows sees: bounds for whole tiles.
struct View {
  int pre_least, pre_most, lo_least, lo_most, hi_least, hi_most;
  // every row sees all of [a, a + n)
  __device__ __forceinline__ bool all(int a, int n) const {
    return (a >= lo_most && hi_least - a >= n) || pre_least - a >= n;
  }
  // some row may see some of [a, a + n)
  __device__ __forceinline__ bool some(int a, int n) const {
    return a < pre_most || (a < hi_most && lo_least - a < n);
  }
};

__device__ __forceinline__ View view_of_wave(const Sight& v) {
  // (rows that see nothing beyond the prefix do not widen the range)
  const bool any = v.hi > v.lo;
  return {wave_min(v.pre), wave_max(v.pre), wave_min(any ? v.lo : INT32_MAX), wave_max(any ? v.lo : INT32_MAX),
          wave_min(any ? v.hi : 0), wave_max(any ? v.hi : 0)};
}

// The quotient of a token and block_tokens.
__device__ __forceinline__ int block_of(const PageAttendParams& p, int token) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(token)) * p.block_magic) >> p.block_shift);
}

// A row of queries as operands.  keep and flip: masks of their bits, which turn
// the sign over where sm_scale is negative and make them 0 where it is 0, so
// that the scale itself is positive.
template <int DT>
struct Queries {
  s8 x[8];
  __device__ __forceinline__ void load(const char* row, int h, uint32_t keep, uint32_t flip) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      u32x4 raw = *reinterpret_cast<const u32x4*>(row + (16 * kk + 8 * h) * 2);
      raw = (raw & keep) ^ flip;
      x[kk] = __builtin_bit_cast(s8, raw);
    }
  }
};
template <>
struct Queries<kF32> {
  f32x4 x[16];
  __device__ __forceinline__ void load(const char* row, int h, uint32_t keep, uint32_t flip) {
#pragma unroll
    for (int kk = 0; kk < 16; ++kk) {
      u32x4 raw = *reinterpret_cast<const u32x4*>(row + (64 * h + 4 * kk) * 4);
      raw = (raw & keep) ^ flip;
      x[kk] = __builtin_bit_cast(f32x4, raw);
    }
  }
};

template <int DT>
__device__ __forceinline__ f32x16 mma(s8 a, s8 b, f32x16 c) {
  if constexpr (DT == kBF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

// A copy of x that the compiler takes for a new value: what is computed from
// it stays where it stands instead of holding registers across a loop.
template <class T>
__device__ __forceinline__ T here(T x) {
  asm volatile("" : "+v"(x));
  return x;
}

// S^T of the subtile's 32 tokens (rows of `keys`, the first a multiple of 32).
template <int DT>
__device__ __forceinline__ f32x16 score_tile(const char* keys, const Queries<DT>& q, int lane) {
  const int id = here(lane);
  const int token = id & 31, h = id >> 5;
  // (a step moves the chunk's place by bits of its own: rows are aligned)
  const int at = token * Row<DT>::kBytes + (Row<DT>::key(token, DT == kF32 ? 16 * h : h) << 4);
  f32x16 acc = {};
  if constexpr (DT == kF32) {
#pragma unroll
    for (int kk = 0; kk < 16; ++kk) {
      const f32x4 k = *reinterpret_cast<const f32x4*>(keys + (at ^ (kk << 4)));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(k[i], q.x[kk][i], acc, 0, 0, 0);
    }
  } else {
    // all reads first, so that the products wait once
    s8 k[8];
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) k[kk] = *reinterpret_cast<const s8*>(keys + (at ^ (kk << 5)));
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) acc = mma<DT>(k[kk], q.x[kk], acc);
  }
  return acc;
}

// Two weights rounded to the type, the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t pack_two(float x, float y) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  if constexpr (DT == kBF16) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{x, y}), b2));
  } else {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{x, y}), h2));
  }
}

// 8 weights as an operand, and (PP = 2) what rounding them left out.
template <int DT, int PP>
struct Weights {
  s8 part[PP][2];
  __device__ __forceinline__ void set(const float (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (DT == kBF16) {
        const __bf16 hi = static_cast<__bf16>(w[i]);
        part[0][i >> 3][i & 7] = __builtin_bit_cast(short, hi);
        if constexpr (PP > 1)
          part[1][i >> 3][i & 7] = __builtin_bit_cast(short, static_cast<__bf16>(w[i] - static_cast<float>(hi)));
      } else {
        const _Float16 hi = static_cast<_Float16>(w[i]);
        part[0][i >> 3][i & 7] = __builtin_bit_cast(short, hi);
        if constexpr (PP > 1)
          part[1][i >> 3][i & 7] = __builtin_bit_cast(short, static_cast<_Float16>(w[i] - static_cast<float>(hi)));
      }
    }
  }
};
template <int PP>
struct Weights<kF32, PP> {
  float w[16];
  __device__ __forceinline__ void set(const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = x[i];
  }
};

typedef __attribute__((address_space(3))) s4* LdsS4;

// O^T += V^T P^T over the subtile's 32 tokens.
template <int DT, int PP>
__device__ __forceinline__ void output_tile(const char* values, const Weights<DT, PP>& w, f32x16 (&o)[4],
                                            int lane) {
  const int id = here(lane);
  const int h = id >> 5;
  if constexpr (DT == kF32) {
    const int dim = id & 31;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int token = 8 * (i >> 2) + 4 * h + (i & 3);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int chunk = 8 * d + (dim >> 2);
        const float v = *reinterpret_cast<const float*>(values + token * Row<DT>::kBytes +
                                                        (Row<DT>::value(token, chunk) << 4) + 4 * (dim & 3));
        o[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(v, w.w[i], o[d], 0, 0, 0);
      }
    }
  } else {
    // A read takes 4 tokens of 16 dims for 16 lanes, lane i supplying the
    // address of token i / 4, dims 4 (i % 4) .., and getting dim i.
    const int i = id & 15;
    const int token = 4 * h + (i >> 2);
    // (d moves the chunk's place by bits of its own)
    const int base = token * Row<DT>::kBytes + (Row<DT>::value(token, 2 * ((id >> 4) & 1) + ((i >> 1) & 1)) << 4) + 8 * (i & 1);
    s8 v[2][4];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const char* at = values + (base ^ (d << 6)) + 16 * s * Row<DT>::kBytes;
        const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS4)(at));
        const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS4)(at + 8 * Row<DT>::kBytes));
        v[s][d] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int pp = PP - 1; pp >= 0; --pp)
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] = mma<DT>(v[s][d], w.part[pp][s], o[d]);
  }
}

// How scores become exponents of two.  Without cap and bias the product is
// scaled in the step that takes the reference off.
struct ScoreScale {
  float scale;       // sm_scale log2(e), or (CAP) sm_scale / cap; positive
  float top;         // (CAP) cap log2(e)
  float slope;       // (BIAS) the head's, times log2(e)
};

// tanh(y): the fraction of exponentials, which loses bits beside 0, or there
// y + y^3 p(y^2), p fitted for the least largest error of the whole, 2^-25 of it.
// NEAR: |y| < kNear (or NaN).
constexpr float kNear = 0.5f;
template <bool NEAR>
__device__ __forceinline__ float tanh_of(float y) {
  const float y2 = y * y;
  float c = __builtin_fmaf(y2, 0.01724161f, -0.05304554f);
  c = __builtin_fmaf(c, y2, 0.13325879f);
  c = __builtin_fmaf(c, y2, -0.33333144f);
  const float small = __builtin_fmaf(y * y2, c, y);
  if constexpr (NEAR) return small;
  const float a = fabsf(y);
  const float e = __builtin_amdgcn_exp2f(-2.88539008177792681472f * a);
  const float big = (1.0f - e) * __builtin_amdgcn_rcpf(1.0f + e);
  return a < kNear ? small : __builtin_copysignf(big, y);
}

template <bool CAP, bool BIAS, bool NEAR>
__device__ __forceinline__ float score_of(float x, const ScoreScale& f, float distance) {
#pragma clang fp contract(off)
  float s = x * f.scale;
  if constexpr (CAP) s = tanh_of<NEAR>(s) * f.top;
  if constexpr (BIAS) s = s - f.slope * distance;
  return s;
}

__device__ __forceinline__ bool is_far(float m) { return fabsf(m) >= kFar && m != kNoReference; }

// State of a wave's rows.
struct RowsState {
  f32x16 o[4];
  float m, l;        // the reference; this lane's part of the sum
  bool far;          // some row's reference is
  float scale, shift;  // of the tile at hand: weights are exp2(scale x + shift)
};

// Bits of the tokens that a row sees of a tile of up to 64 from `first` on, of
// which `live` exist, bit 0 that of register 0.
__device__ __forceinline__ uint64_t seen_of(const Sight& v, uint64_t live, int first, int h) {
  auto below = [&](int end) {            // tokens before `end`
    const int n = min(max(end - first, 0), 64);
    return n == 64 ? ~uint64_t{0} : (uint64_t{1} << n) - 1;
  };
  return (live & (below(v.pre) | (below(v.hi) & ~below(v.lo)))) >> (4 * h);
}

// The largest of a tile's products, once the scores are made of them that have
// a cap or a bias (the others stay products).  from_first: the row's position,
// counted from the token of register 0.
// Scores below half their cap, as they mostly are, need the polynomial alone,
// which is less than half the work: 1,229 rows over 8,192 tokens of a reordered
// context, capped at 30, take 157 us, 187 with both (129 without a cap).
template <bool CAP, bool BIAS, int N>
__device__ __forceinline__ float scores_of(f32x16 (&acc)[N], const ScoreScale& f, float from_first) {
  if constexpr (CAP || BIAS) {
    auto make = [&](auto near) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < N; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          // (kept from being made ahead of the choice)
          const float x = CAP && !decltype(near)::value ? here(acc[u][i]) : acc[u][i];
          acc[u][i] = score_of<CAP, BIAS, decltype(near)::value>(x, f, fabsf(from_first - (kSub * u + 8 * (i >> 2) + (i & 3))));
        }
    };
    float most = 0.0f;
    if constexpr (CAP) {
#pragma unroll
      for (int u = 0; u < N; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(acc[u][i]));
    }
    if (CAP && __all(most * f.scale < kNear))
      make(std::true_type{});
    else
      make(std::false_type{});
  }
  float top = -INFINITY;
#pragma unroll
  for (int u = 0; u < N; ++u)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, acc[u][i]);
  return top;
}

// Masks a tile's scores (part: some row may not see all of it; seen: what the
// lane's row sees of it, see seen_of), moves the reference where they outgrow it
// and says how they become weights.
template <int DT, bool CAP, bool BIAS, int N>
__device__ __forceinline__ void refer_tile(f32x16 (&acc)[N], float top, RowsState& st, const ScoreScale& f,
                                           bool part, uint64_t seen) {
  constexpr float kOff = PageTraits<DT>::kOff, kSlack = PageTraits<DT>::kSlack;
  constexpr bool kPlain = !CAP && !BIAS;
  if (part) {
    top = -INFINITY;
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        acc[u][i] = (seen >> (kSub * u + 8 * (i >> 2) + (i & 3))) & 1 ? acc[u][i] : -INFINITY;
        top = fmaxf(top, acc[u][i]);
      }
  }
  if constexpr (kPlain) top *= f.scale;            // (scale > 0)
  if (__any(top > st.m + kSlack)) {
    top = fmaxf(top, __shfl_xor(top, 32));
    const float m = top > st.m + kSlack ? ceilf(top) : st.m;
    const float keep = m == st.m ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
    st.m = m;
    st.l *= keep;
#pragma unroll
    for (int d = 0; d < 4; ++d) st.o[d] *= keep;
    st.far = __any(is_far(m));
  }
  st.scale = kPlain ? f.scale : 1.0f;
  st.shift = kOff - st.m;
  if (st.far) {
    // A far reference came from rounded scores: so do the row's weights.  And it is
    // taken off by itself: beside a reference from 2^26 on kOff is lost in the
    // shift.  (Rows whose own reference is near keep their one rounding.)
#pragma clang fp contract(off)
    const bool far = is_far(st.m);
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float away = (kPlain ? acc[u][i] * f.scale : acc[u][i]) - st.m;
        acc[u][i] = far ? away : acc[u][i];
      }
    st.scale = far ? 1.0f : st.scale;
    st.shift = far ? kOff : st.shift;
  }
}

// The weights of a subtile and their sum.
template <int DT, int PP>
__device__ __forceinline__ float weigh_tile(const f32x16& acc, Weights<DT, PP>& out, const RowsState& st) {
  float w[16], sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i], st.scale, st.shift));
    sum += w[i];
  }
  out.set(w);
  return sum;
}

// 16 bytes per lane straight into LDS: lane i's to `to` + 16 i.
__device__ __forceinline__ void bring16(const char* from, char* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t*)(from),
                                   (__attribute__((address_space(3))) uint32_t*)(to), 16, 0, 0);
}

// What a wave brings at once: the keys or values of a group of tokens, 4 loads.
// In LDS they lie as in Row; the first token of a group is a multiple of kTokens.
template <int DT>
struct Group {
  using R = Row<DT>;
  static constexpr int kLoads = 4;
  static constexpr int kTokens = kLoads * R::kPerWave;

  // This lane's part of a load of a whole group: its row's offset, and its
  // chunk's place, which load n moves by bits of its own.
  struct Lane {
    uint32_t row_off, place;
    __device__ __forceinline__ Lane(const PageAttendParams& p, bool key, int first, int lane) {
      const int row = lane / R::kChunks, chunk = lane % R::kChunks;
      row_off = static_cast<uint32_t>(row) * static_cast<uint32_t>(p.token);
      place = (key ? R::key(first + row, chunk) : R::value(first + row, chunk)) << 4;
    }
  };
  static __device__ __forceinline__ uint32_t turn(bool key, int n) {
    return 16 * (key ? R::kPerWave * n : R::value(R::kPerWave * n, 0));
  }
  // Load n; `rows` is the first of the group's tokens.
  static __device__ __forceinline__ void bring_one(const PageAttendParams& p, const char* rows, const Lane& lane, bool key,
                                                   int n, char* to) {
    const uint32_t off = here(lane.row_off) + (here(lane.place) ^ turn(key, n));
    bring16(rows + n * (R::kPerWave * p.token) + off, to + 16 * kWave * n);
  }

  // Groups whose tokens lie apart or do not all exist: `at` is the place of
  // token lane % kTokens, -1 if it does not exist.
  static __device__ __forceinline__ int64_t place(const PageAttendParams& p, int token, int len, int entry, int64_t head_off) {
    const bool known = token < len && static_cast<uint32_t>(entry) < static_cast<uint32_t>(p.num_pages);
    return known ? entry * p.page + (token - block_of(p, token) * p.block_tokens) * p.token + head_off : int64_t{-1};
  }
  static __device__ __forceinline__ void bring_apart(const char* from, int64_t at, bool key, int first, char* to, int lane) {
    const int row = lane / R::kChunks, chunk = lane % R::kChunks;
    const char* none = reinterpret_cast<const char*>(kZeros);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int t = R::kPerWave * n + row;
      const int64_t off = __shfl(at, t);
      bring16(off < 0 ? none : from + off + ((key ? R::key(first + t, chunk) : R::value(first + t, chunk)) << 4),
              to + 16 * kWave * n);
    }
  }
};

// Waits until at most N of the wave's loads are under way (they arrive in
// order), and for its LDS reads.  Nothing moves across.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "vmcnt has 6 bits");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"(N) : "memory");
}

// log(2^m l), m a whole number; -infinity for l = 0.
__device__ __forceinline__ float lse_of(float m, float l) {
  const int e = l > 0.0f && l < INFINITY ? __builtin_amdgcn_frexp_expf(l) : 0;
  return (__builtin_amdgcn_logf(__builtin_ldexpf(l, -e)) + (m + static_cast<float>(e))) * kLn2;
}

// The tiles that a wave has worked on: first, first + step, .. of a list.
struct WaveTiles {
  TileList list;
  int first, end, step, size;
};

// What of a type is not finite: all bits of its exponent are set.
template <int DT>
__device__ __forceinline__ bool not_finite(uint32_t bits) {
  constexpr uint32_t kExponent = DT == kF32 ? 0x7F800000u : DT == kF16 ? 0x7C00u : 0x7F80u;
  return (bits & kExponent) == kExponent;
}

// 4 consecutive elements as fp32.
template <int DT>
__device__ __forceinline__ f32x4 load4(const char* from) {
  if constexpr (DT == kF32) {
    return *reinterpret_cast<const f32x4*>(from);
  } else {
    const u32x2 raw = *reinterpret_cast<const u32x2*>(from);
    f32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t bits = (raw[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
      y[i] = DT == kF16 ? f16_bits_to_f32(bits) : bf16_bits_to_f32(bits);
    }
    return y;
  }
}

// How far weights are made smaller where the output is made again, so that sums
// of up to 2^31 of them (each 2^kSlack at most) times the type's largest values
// stay in fp32's range, before the weights' sum is divided out.  (fp16's values
// leave room; weights below 2^-126 of this lose bits, 2^-86 of a row's largest.)
template <int DT> constexpr float kSmaller = DT == kF16 ? 1.0f : 0x1p-40f;

// O^T over a wave's tiles once more, N subtiles each, for values that are not
// finite or too large: the same products, references and weights in the same
// order, so that a row has the same bits whatever the tokens hold that it does not
// see, but from the pages and with every value that is not finite taken as 0.
// Those are added by themselves to the rows where their token has a weight above 0.
// Out of the way of the common case: no LDS, 2-byte loads and a wait at each step
// (one token of NaN in 4,096 that all rows see: 512 queries of 32 heads take 440 us
// for 60, a decode 30 for 18).
template <int DT, int PP, bool CAP, bool BIAS, int N>
__device__ __forceinline__ void output_again(const PageAttendParams& p, const int32_t* table, int64_t head_off,
                                             const char* q_row, const Sight& v, int len, const WaveTiles& w,
                                             const ScoreScale& f, f32x16 (&o)[4], int lane) {
  constexpr int ES = ElemSize<DT>::value;
  const char* none = reinterpret_cast<const char*>(kZeros);
  const int q32 = lane & 31, h = lane >> 5;
  Queries<DT> q;
  // (as scalars of their own: loaded together with their neighbours they put those
  // parameters into scratch memory for the whole kernel)
  q.load(q_row, h, __builtin_amdgcn_readfirstlane(p.q_keep), __builtin_amdgcn_readfirstlane(p.q_flip));
  RowsState st;
#pragma unroll
  for (int d = 0; d < 4; ++d) st.o[d] = f32x16{};
  st.m = kNoReference;
  st.l = 0.0f;
  st.far = false;
  for (int i = w.first; i < w.end; i += w.step) {
    const int first = w.list.at(i) * w.size;
    int64_t at[N];                       // places of tokens lane % 32 of the subtiles
    uint64_t live = 0;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int token = first + kSub * u + q32;
      const int block = block_of(p, token);
      const int entry = token < len ? table[block] : -1;
      const bool known = static_cast<uint32_t>(entry) < static_cast<uint32_t>(p.num_pages);
      at[u] = known ? entry * p.page + (token - block * p.block_tokens) * p.token + head_off : int64_t{-1};
      live |= static_cast<uint64_t>(static_cast<uint32_t>(__ballot(known))) << (kSub * u);
    }
    const uint64_t seen = seen_of(v, live, first, h);
    if (!__any(seen != 0)) continue;
    f32x16 acc[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      acc[u] = f32x16{};
      const char* key = p.k + at[u];
      if constexpr (DT == kF32) {
#pragma unroll
        for (int kk = 0; kk < 16; ++kk) {
          const f32x4 k = *reinterpret_cast<const f32x4*>(at[u] < 0 ? none : key + (64 * h + 4 * kk) * ES);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[u] = __builtin_amdgcn_mfma_f32_32x32x2f32(k[e], q.x[kk][e], acc[u], 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          acc[u] = mma<DT>(*reinterpret_cast<const s8*>(at[u] < 0 ? none : key + (16 * kk + 8 * h) * ES), q.x[kk], acc[u]);
      }
    }
    const float from_first = BIAS ? static_cast<float>(static_cast<double>(v.pos) - (first + 4 * h)) : 0.0f;
    const float top = scores_of<CAP, BIAS, N>(acc, f, from_first);
    refer_tile<DT, CAP, BIAS, N>(acc, top, st, f, true, seen);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      float weight[16], smaller[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        weight[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[u][e], st.scale, st.shift));
        smaller[e] = weight[e] * kSmaller<DT>;
      }
      Weights<DT, PP> operand;
      operand.set(smaller);
      uint32_t odd = 0;                  // tokens with a value that is not finite
#pragma unroll
      for (int s = 0; s < 2; ++s) {      // (halves by themselves: fewer registers)
        __builtin_amdgcn_sched_barrier(0);
        s8 x[4];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int t = 16 * s + 8 * (e >> 2) + (e & 3);
          const int64_t place = __shfl(at[u], t + 4 * h);
          const char* value = place < 0 ? none : p.v + place + q32 * ES;
          const int step = place < 0 ? 0 : 32 * ES;
          bool bad = false;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            if constexpr (DT == kF32) {
              const uint32_t bits = *reinterpret_cast<const uint32_t*>(value + d * step);
              const bool is = not_finite<DT>(bits);
              bad = bad || is;
              st.o[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(is ? 0.0f : __builtin_bit_cast(float, bits),
                                                             operand.w[8 * s + e], st.o[d], 0, 0, 0);
            } else {
              const uint16_t bits = *reinterpret_cast<const uint16_t*>(value + d * step);
              const bool is = not_finite<DT>(bits);
              bad = bad || is;
              x[d][e] = is ? 0 : static_cast<short>(bits);
            }
          }
          const uint64_t all = __ballot(bad);
          odd |= static_cast<uint32_t>(static_cast<uint32_t>(all) != 0) << t |
                 static_cast<uint32_t>((all >> 32) != 0) << (t + 4);
        }
        if constexpr (DT != kF32) {
#pragma unroll
          for (int pp = PP - 1; pp >= 0; --pp)
#pragma unroll
            for (int d = 0; d < 4; ++d) st.o[d] = mma<DT>(x[d], operand.part[pp][s], st.o[d]);
        }
      }
      while (odd) {
        const int t = __builtin_ctz(odd);
        odd &= odd - 1;
        float mine = 0.0f;               // token t's weight, in the lanes that have it
#pragma unroll
        for (int e = 0; e < 16; ++e) mine = 8 * (e >> 2) + (e & 3) == (t & ~4) ? weight[e] : mine;
        const float that = __shfl(mine, q32 + 8 * (t & 4));
        const char* value = p.v + __shfl(at[u], t) + 4 * h * ES;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const f32x4 y = load4<DT>(value + (32 * d + 8 * a) * ES);
#pragma unroll
            for (int b = 0; b < 4; ++b)
              st.o[d][4 * a + b] += that > 0.0f && !(fabsf(y[b]) < INFINITY) ? that * y[b] : 0.0f;
          }
      }
    }
  }
#pragma unroll
  for (int d = 0; d < 4; ++d) o[d] = st.o[d];
}

// Divides the sum out (l becomes the row's whole sum of this wave's tokens), of
// an output that is made again where some row's is not finite.
template <int DT, int PP, bool CAP, bool BIAS, int N>
__device__ __forceinline__ void finish_rows(const PageAttendParams& p, const int32_t* table, int64_t head_off,
                                            const char* q_row, const Sight& v, int len, const WaveTiles& w,
                                            RowsState& st, const ScoreScale& f, int lane) {
  st.l += __shfl_xor(st.l, 32);
  float inv = 1.0f / st.l;
  bool bad = false;
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) bad = bad || !(fabsf(st.o[d][i] * inv) < INFINITY);
  if (__any(bad && st.l > 0.0f && st.l < INFINITY)) {
    output_again<DT, PP, CAP, BIAS, N>(p, table, head_off, q_row, v, len, w, f, st.o, lane);
    inv *= 1.0f / kSmaller<DT>;
  }
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) st.o[d][i] = st.l == 0.0f ? 0.0f : st.o[d][i] * inv;
  st.l *= __builtin_amdgcn_exp2f(-PageTraits<DT>::kOff);
}

// 4 consecutive dims of a row.
template <int DT>
__device__ __forceinline__ void store4(char* p, const float (&x)[4]) {
  if constexpr (DT == kF32) {
    *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
  } else {
    u32x2 y;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = DT == kF16 ? f32_to_f16_bits(x[2 * i]) : f32_to_bf16_bits(x[2 * i]);
      const uint32_t hi = DT == kF16 ? f32_to_f16_bits(x[2 * i + 1]) : f32_to_bf16_bits(x[2 * i + 1]);
      y[i] = lo | (hi << 16);
    }
    *reinterpret_cast<u32x2*>(p) = y;
  }
}

// The slope and scales of a head's rows.
template <bool BIAS>
__device__ __forceinline__ ScoreScale scale_of(const PageAttendParams& p, int head) {
  return {p.scale, p.cap_log2, BIAS ? p.slopes[head] * 1.44269504088896340736f : 0.0f};
}

}  // namespace hkv
