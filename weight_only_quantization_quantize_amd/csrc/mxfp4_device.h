// Device helpers of the microscaled 4-bit float (MXFP4) kernels.
//
// Format.  32 consecutive elements of a row share one scale byte b standing
// for 2^(b - 127) (b = 255: the block is not a number); an element is a 4-bit
// float e2m1 (sign, then 0 0.5 1 1.5 2 3 4 6), two per byte, even k in the low
// nibble.  One block is 16 bytes of codes, which is exactly what one lane of
// v_mfma_scale_f32_{16x16x128,32x32x64}_f8f6f4 supplies, with one scale byte:
// the stored format is the matrix units' own operand format.
#pragma once

#include "woq_device.h"

namespace woq {

constexpr int kMxBlock = 32;      // elements per scale
constexpr int kMxNan = 255;       // scale byte of a block that is not a number

typedef float float16_t __attribute__((ext_vector_type(16)));
typedef float float2_t __attribute__((ext_vector_type(2)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Operand format selector of the scaled matrix instructions: e2m1.
constexpr int kMfmaFp4 = 4;

// 2^(b - 127) for b in [0, 254]; a quiet NaN for 255.
__device__ inline float mx_pow2(uint32_t b) {
  const uint32_t bits = b == 0 ? 0x00400000u : (b << 23);
  return __builtin_bit_cast(float, b == (uint32_t)kMxNan ? 0x7FC00000u : bits);
}

// Scale byte of a block whose largest magnitude is amax: the exponent of amax
// less 2, the exponent of the largest element value 6 (so amax / scale lies in
// [4, 8) and what exceeds 6 saturates), held to [0, 254].  A zero block gives
// 0 and one with an infinity or a NaN gives 255.
__device__ inline uint32_t mx_scale_byte(float amax) {
  const uint32_t e = __builtin_bit_cast(uint32_t, amax) >> 23;  // 0 for zero and fp32-subnormal magnitudes
  return e == 255u ? (uint32_t)kMxNan : (e > 2u ? e - 2u : 0u);
}

// The larger of two magnitudes, a NaN if either is one.
__device__ inline float mx_absmax(float a, float b) {
  const uint32_t x = __builtin_bit_cast(uint32_t, a) & 0x7FFFFFFFu, y = __builtin_bit_cast(uint32_t, b) & 0x7FFFFFFFu;
  return __builtin_bit_cast(float, x > y ? x : y);
}

__device__ inline i32x8_t mx_operand(u32x4_t v) {
  return i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

// 16-bit activations by microscaled weights.  The activations are used as they are,
// and a weight is widened to their type: one conversion makes two codes c 2^(b - 127)
// for the 16-bit matrix instructions (exact products, fp32 sums; subnormal operands
// and sums are kept).  No operand is rounded.
//   bf16  a quarter of the weights, so that none is too large; the sums are multiplied
//         by kMxGain.  Scale bytes 0, 1 and 255 take a slower way to the same.
//   fp16  holds the weights of scale bytes 104 .. 140.  A wave that meets others
//         multiplies that step in bf16 (mx_general_*): the activations as the sum of
//         two numbers, their 11 bits in 8 and 3, and weights that may be 2^128 and
//         more as four equal parts.
template <class XT>
constexpr bool kMxIsF16 = XT::kMagic2 == F16::kMagic2;
template <class XT>
constexpr float kMxGain = kMxIsF16<XT> ? 1.0f : 4.0f;

// Whether one of the low `n` bytes of `scales` may need the slower way.  fp16: held to
// 104 .. 135, which a subtraction over all bytes tells: where a byte is below 104 the
// borrow changes the next one, but its own top bits show it.  bf16: 255, 0, 1 (and 2)
// are those that 1 more brings below 4.
template <class XT>
__device__ inline bool mx_unusual(uint32_t scales, int n) {
  const uint32_t bytes = n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
  if constexpr (kMxIsF16<XT>) return ((scales - (0x68686868u & bytes)) & (0xE0E0E0E0u & bytes)) != 0;
  const uint32_t t = (scales + 0x01010101u) & 0xFCFCFCFCu;
  return ((t - 0x01010101u) & ~t & 0x80808080u & bytes) != 0;
}
// Whether a block of codes c at scale byte b needs it: zeros do not, but at 255 and, in
// bf16, at 1, of which mx_widen would make it.
template <class XT>
__device__ inline bool mx_needs_care(u32x4_t c, uint32_t b) {
  return mx_unusual<XT>(b, 1) &&
         (((c[0] | c[1] | c[2] | c[3]) & 0x77777777u) != 0 || b == (uint32_t)kMxNan || (!kMxIsF16<XT> && b == 1u));
}

// The 8 weights of a dword of codes at scale byte b (255: NaNs).
template <class XT>
__device__ inline u32x4_t mx_widen_as_is(uint32_t c, uint32_t b) {
  const float s = __builtin_bit_cast(float, b << 23);  // the conversion reads the exponent bits, 0 as 2^-127
  if constexpr (kMxIsF16<XT>)
    return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 0)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 1)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 2)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 3))};
  else
    return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3))};
}
// The same over kMxGain, for scale bytes that mx_needs_care is false for.
template <class XT>
__device__ inline u32x4_t mx_widen(uint32_t c, uint32_t b) {
  return mx_widen_as_is<XT>(c, kMxIsF16<XT> ? b : b - 2u);
}
// bf16, any scale byte: the few low ones through fp32, where their quarters are exact.
__device__ __forceinline__ u32x4_t mx_widen_any(uint32_t c, uint32_t b) {
  asm volatile("" : "+v"(c));  // worked out here: kept for later, it spills
  const bool low = b < 2u;
  u32x4_t w = mx_widen_as_is<BF16>(c, low || b == (uint32_t)kMxNan ? b : b - 2u);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float x = __builtin_bit_cast(float, w[e] << 16) * 0.25f, y = __builtin_bit_cast(float, w[e] & 0xFFFF0000u) * 0.25f;
    const uint32_t q = __builtin_bit_cast(uint32_t, x) >> 16 | (__builtin_bit_cast(uint32_t, y) & 0xFFFF0000u);
    w[e] = low ? q : w[e];
  }
  return w;
}

// fp16, the general step: kMxPasses products (every fourth where no lane of the wave
// has weights that may be 2^128 or more), each of mx_general_weights and
// mx_general_activations of the same number, in bf16.
constexpr int kMxPasses = 8;
__device__ inline bool mx_large(uint32_t b) { return b == 253u || b == 254u; }
// The weights of passes 0 and 4; a quarter in each pass where they may be large.
__device__ __forceinline__ u32x4_t mx_general_weights(uint32_t c, uint32_t b, int pass) {
  asm volatile("" : "+v"(c));  // worked out where it is used: kept for all passes, it spills
  const bool large = mx_large(b);
  const u32x4_t w = mx_widen_as_is<BF16>(c, large ? b - 2u : b);
  return large || (pass & 3) == 0 ? w : u32x4_t{0u, 0u, 0u, 0u};
}
// Eight activations' high (passes 0 .. 3) or low part.  What is not finite counts
// once: in pass 0.
__device__ __forceinline__ u32x4_t mx_general_activations(u32x4_t x, int pass) {
  u32x4_t r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t out = 0, pair = x[e];
    asm volatile("" : "+v"(pair));  // as above
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float v = F16::to_f32((uint16_t)(pair >> (16 * h)));
      const uint16_t high = BF16::from_f32(v);
      const uint16_t part = pass < 4 ? high : BF16::from_f32(v - BF16::to_f32(high));
      const bool finite = (high & 0x7F80u) != 0x7F80u;
      out |= (uint32_t)(finite || pass == 0 ? part : (uint16_t)0) << (16 * h);
    }
    r[e] = out;
  }
  return r;
}

template <class XT>
__device__ inline float16_t mfma32x32x16(u32x4_t a, u32x4_t b, float16_t c) {
  if constexpr (kMxIsF16<XT>)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf168_t, a), __builtin_bit_cast(bf168_t, b), c, 0, 0, 0);
}

// Fragment-major storage of activations.  A fragment is R rows (32 or 16) by
// 2048 / R elements of K (2 or 4 blocks): lane l of a wave holds row l % R, block
// l / R, 16 bytes (8 elements) of every lane after 16 bytes of every lane.
// Fragments lie [row group][K step], rows past M and blocks past K are zeros.
// With R = 16 four steps make a super-step of 16 blocks, and lane group l / 16
// holds block 4 (l / 16) + s of it at its step s.
constexpr int kMxFragBytes = 64 * 64;

// Scale bytes 16 g .. 16 g + 15 of a row of nblk, `past` behind its end, in each
// dword in the order 0, 2, 1, 3.
__device__ inline u32x4_t mx_scale_chunk(const uint8_t* __restrict__ row, int g, int nblk, uint32_t past) {
  u32x4_t v = {0u, 0u, 0u, 0u};
  const uint8_t* const p = row + 16 * g;
  if (16 * g + 16 <= nblk) {
    __builtin_memcpy(&v, p, 16);
  } else {
#pragma unroll
    for (int q = 0; q < 16; ++q)
      v[q / 4] |= (16 * g + q < nblk ? (uint32_t)p[q] : past) << (8 * (q % 4));
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = __builtin_amdgcn_perm(v[q], v[q], 0x03010200u);
  return v;
}

}  // namespace woq
