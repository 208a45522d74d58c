// Device code of the quantizer shared by the put (quant.hip) and the token
// append (append.hip): one vector's scale, codes and their stores.
#pragma once

#include "hkv_device.h"

namespace hkv {

// fp16 bits of the scale for a vector with max magnitude amax (fp32).
// Edge cases: amax == 0 -> 0; a positive amax whose scale underflows fp16 ->
// smallest subnormal (0x0001); a scale beyond the fp16 range -> 65504.
template <int QMAX>
__device__ __forceinline__ uint32_t scale_bits(float amax) {
  const float s32 = amax / static_cast<float>(QMAX);   // IEEE division
  uint32_t h = f32_to_f16_bits(s32);
  if (h == 0x7C00u) h = 0x7BFFu;
  if (h == 0u && amax > 0.0f) h = 0x0001u;
  return h;
}

// Source run of 8 elements (lane-owned half of a vector) as raw words.
template <int SDT> struct RawSrc;
template <> struct RawSrc<kF32> { u32x4 w0, w1; };
template <> struct RawSrc<kF16> { u32x4 w0; };
template <> struct RawSrc<kBF16> { u32x4 w0; };

template <int SDT>
__device__ __forceinline__ RawSrc<SDT> load_run(const char* p) {
  RawSrc<SDT> r;
  r.w0 = *reinterpret_cast<const u32x4*>(p);
  if constexpr (SDT == kF32) r.w1 = *reinterpret_cast<const u32x4*>(p + 16);
  return r;
}

template <int SDT>
__device__ __forceinline__ void run_to_f32(const RawSrc<SDT>& r, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = r.w0[j];
    if constexpr (SDT == kF32) {
      const uint32_t w1 = r.w1[j];
      x[j] = __builtin_bit_cast(float, w);
      x[4 + j] = __builtin_bit_cast(float, w1);
    } else if constexpr (SDT == kF16) {
      x[2 * j] = f16_bits_to_f32(w & 0xFFFFu);
      x[2 * j + 1] = f16_bits_to_f32(w >> 16);
    } else {
      x[2 * j] = bf16_bits_to_f32(w & 0xFFFFu);
      x[2 * j + 1] = bf16_bits_to_f32(w >> 16);
    }
  }
}

// Quantize one vector's lane-owned runs a (elements 8s..8s+7) and b
// (64+8s..64+8s+7); returns the fp16 scale bits (same in all 8 lanes).
// STAGE: the code bytes also go to `stage` (LDS) at the same offsets.
template <int FMT, bool STAGE>
__device__ __forceinline__ uint32_t quant_vector(float (&a)[8], float (&b)[8], uint8_t* c_ptr,
                                                 int sub, bool active, uint8_t* stage) {
  // |x| compared as integers: for finite values the magnitude bits order
  // exactly like the magnitudes.
  uint32_t mbits = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t ua = __builtin_bit_cast(uint32_t, a[j]) & 0x7FFFFFFFu;
    const uint32_t ub = __builtin_bit_cast(uint32_t, b[j]) & 0x7FFFFFFFu;
    mbits = max(mbits, max(ua, ub));
  }
  const float amax = __builtin_bit_cast(float, max_bits_over_vector_lanes(mbits));
  constexpr int QMAX = FMT == kFP8 ? 448 : 7;
  const uint32_t sbits = scale_bits<QMAX>(amax);
  if (!active) return sbits;
  // An all-zero vector (s = 0) keeps its signed zeros: divide by 1 instead.
  const float s = sbits == 0u ? 1.0f : f16_bits_to_f32(sbits);
  const float r = 1.0f / s;                              // IEEE division, once per vector
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    a[j] = div_by_scale(a[j], s, r);
    b[j] = div_by_scale(b[j], s, r);
  }
  if constexpr (FMT == kFP8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] = __builtin_amdgcn_fmed3f(a[j], -448.0f, 448.0f);
      b[j] = __builtin_amdgcn_fmed3f(b[j], -448.0f, 448.0f);
    }
    const u32x2 ca = f32x8_to_fp8(a);
    const u32x2 cb = f32x8_to_fp8(b);
    __builtin_nontemporal_store(ca, reinterpret_cast<u32x2*>(c_ptr + 8 * sub));
    __builtin_nontemporal_store(cb, reinterpret_cast<u32x2*>(c_ptr + 64 + 8 * sub));
    if constexpr (STAGE) {
      *reinterpret_cast<u32x2*>(stage + 8 * sub) = ca;
      *reinterpret_cast<u32x2*>(stage + 64 + 8 * sub) = cb;
    }
  } else {
    // q clamped to [-7, 7] (integers, so clamping before rounding is the
    // same as after), then 1.5 * 2^23 added: the fp32 sum has unit spacing
    // there, so the addition itself rounds q to the nearest integer, ties
    // to even, and the low four bits of the sum are that integer in two's
    // complement -- the nibble.
    uint32_t wa = 0, wb = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float ra = __builtin_amdgcn_fmed3f(a[j], -7.0f, 7.0f) + 12582912.0f;
      const float rb = __builtin_amdgcn_fmed3f(b[j], -7.0f, 7.0f) + 12582912.0f;
      wa |= (__builtin_bit_cast(uint32_t, ra) & 0xFu) << (4 * j);
      wb |= (__builtin_bit_cast(uint32_t, rb) & 0xFu) << (4 * j);
    }
    __builtin_nontemporal_store(wa, reinterpret_cast<uint32_t*>(c_ptr + 4 * sub));
    __builtin_nontemporal_store(wb, reinterpret_cast<uint32_t*>(c_ptr + 32 + 4 * sub));
    if constexpr (STAGE) {
      *reinterpret_cast<uint32_t*>(stage + 4 * sub) = wa;
      *reinterpret_cast<uint32_t*>(stage + 32 + 4 * sub) = wb;
    }
  }
  return sbits;
}

}  // namespace hkv
