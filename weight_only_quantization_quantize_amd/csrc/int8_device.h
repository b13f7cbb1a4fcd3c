// What the 8-bit integer kernels share: the rounding of a row's elements to codes,
// element types, and a row's largest magnitude.
//
// A row y is held as codes q in -127 .. 127 and a scale a / 127, a = max|y|:
//   q = the integer nearest to 127 y / a, ties to the even one, decided exactly.
// y r with r = fl(127 / a) is off by at most 127 2^-24 < 2^-17 (and 2^-18 more where it is
// rounded), so it decides every element but those within kNear of a tie; there the sign of
// 254 |y| - (2 floor(|y| r) + 1) a decides.  Both products are exact as a float and its error
// term (fmaf), their difference next to a tie is exact too, and 0 only at a tie.
#pragma once

#include <type_traits>

#include "woq_device.h"

namespace woq {

typedef int int16v_t __attribute__((ext_vector_type(16)));
typedef int int4v_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// fp32 as an element type, beside F16 and BF16 (woq_device.h).
struct F32 {};
template <class XT>
constexpr int kElementBytes = std::is_same_v<XT, F32> ? 4 : 2;

// An output element of type YT.
template <class YT>
struct Int8Out {
  typedef uint16_t type;
  __device__ static uint16_t of(float v) { return YT::from_f32(v); }
};
template <>
struct Int8Out<F32> {
  typedef float type;
  __device__ static float of(float v) { return v; }
};

// A row's numbers for its codes: from the largest magnitude's bits (of an infinity or a
// NaN: spoilt, scale NaN and codes 0; of a row of zeros: scale 0 and codes 0).
struct Int8Row {
  float factor;  // a power of two that keeps the products below inside fp32's range
  float a, r;    // of y times the factor
  float scale;
};
__device__ inline Int8Row int8_row(uint32_t bits) {
  bits = (uint32_t)__builtin_amdgcn_readfirstlane((int)bits);
  const float a = __builtin_bit_cast(float, bits);
  Int8Row p;
  p.factor = a < 0x1p-60f ? 0x1p80f : (a > 0x1p60f ? 0x1p-80f : 1.0f);
  p.a = a * p.factor;
  p.r = 127.0f / p.a;
  p.scale = a / 127.0f;
  if (bits == 0u || bits >= 0x7F800000u) {
    p.factor = p.a = p.r = 0.0f;
    p.scale = bits == 0u ? 0.0f : __builtin_bit_cast(float, 0x7FC00000u);
  }
  return p;
}

constexpr float kNear = 0x1p-14f;
constexpr float kWhole = 0x1.8p23f;  // adding it rounds to an integer, ties to even, in the low bits

// The codes of N elements of a row, four in a word, the first in the low byte.  The row is
// one for all lanes of the wave.
template <int N>
__device__ inline void int8_codes(const float (&y)[N], const Int8Row& p, uint32_t (&q)[N / 4]) {
  static_assert(N % 4 == 0);
  if (p.r == 0.0f) {  // spoilt, or zeros
#pragma unroll
    for (int i = 0; i < N / 4; ++i) q[i] = 0u;
    return;
  }
  float v[N], z[N], far = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = y[i];
  if (p.factor != 1.0f)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= p.factor;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    z[i] = fmaf(v[i], p.r, kWhole);
    far = fmaxf(far, fabsf(fmaf(v[i], p.r, -(z[i] - kWhole))));
  }
  if (__any(far > 0.5f - kNear)) {
#pragma clang fp contract(off)  // f and s are the rounded products
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float u = fabsf(v[i]), t = u * p.r, low = floorf(t), h = 2.0f * low + 1.0f;
      const float f = 254.0f * u, s = h * p.a;
      const float d = (f - s) + (fmaf(254.0f, u, -f) - fmaf(h, p.a, -s));
      const float even = 2.0f * rintf(0.5f * low + 0.25f);  // the even one of low, low + 1
      const float c = d > 0.0f ? low + 1.0f : (d < 0.0f ? low : even);
      const bool tie = fabsf(t - low - 0.5f) < 2.0f * kNear;
      z[i] = tie ? copysignf(c, v[i]) + kWhole : z[i];
    }
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    auto bits = [&](int k) { return __builtin_bit_cast(uint32_t, z[4 * i + k]); };
    q[i] = __builtin_amdgcn_perm(bits(1), bits(0), 0x0C0C0400u) | __builtin_amdgcn_perm(bits(3), bits(2), 0x04000C0Cu);
  }
}

// silu(g) u
__device__ inline float int8_gated(float g, float u) { return g / (1.0f + expf(-g)) * u; }

__device__ inline uint32_t magnitude(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }
__device__ inline uint32_t wave_max_bits(uint32_t v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, off, 64);
    v = v > o ? v : o;
  }
  return v;
}

}  // namespace woq
