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
constexpr int kMxPieces = 3;      // 6-bit pieces an activation is split into
constexpr int kMxPieceShift[kMxPieces] = {0, 4, 9};  // scale exponents of the pieces, below the first's
constexpr int kMxMinSplit = 10;   // smallest scale byte of the first piece (the third's stays above 0)

typedef float float2_t __attribute__((ext_vector_type(2)));
typedef float float16_t __attribute__((ext_vector_type(16)));
typedef float float32_t __attribute__((ext_vector_type(32)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x6_t __attribute__((ext_vector_type(6)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Operand format selectors of the scaled matrix instructions.
constexpr int kMfmaFp6 = 2;  // e2m3
constexpr int kMfmaFp4 = 4;  // e2m1

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
__device__ inline i32x8_t mx_operand(u32x4_t v, u32x2_t w) {
  return i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], (int)w[0], (int)w[1], 0, 0};
}

// The 6-bit pieces of the activations.  v_mfma_scale takes 4-bit weights
// against 6-bit floats e2m3 (4 significant bits, largest 7.5) at the 4-bit
// rate, so 16-bit activations are multiplied as a sum of three such pieces
//   x = s p1 + (s / 16) p2 + (s / 512) p3 + r
// with s a power of two for each block of 32.  s puts the block's largest
// magnitude in (3.75, 7.5] s; each piece is the nearest e2m3 value to what the
// earlier ones leave: |x - s p1| <= s / 4, then <= (s / 16) / 8, and at last
// |r| <= (s / 512) / 8 = s 2^-12 < 2^-13.9 of the block's largest magnitude.
// fp16 rounds a value to 2^-11 of itself, so at the magnitudes that carry a
// block's sum the pieces hold more than the 16-bit types' own significands
// hold; three matrix steps at the 4-bit rate take 3/4 of a 16-bit one's time
// and the weights are never decoded.
struct MxPieces {
  u32x6_t p[kMxPieces];
  uint32_t scale;  // bytes: the three pieces' scales, 0
};

// The 32-element conversions between fp32 and e2m3 take several passes, and the
// compiler's builtins let their result share registers with a source that a
// later pass still reads (seen in its output, with wrong third pieces); written
// out, the result is a register range of its own.
// Elements 2i come from lo, 2i + 1 from hi.
__device__ inline u32x6_t to_fp6x32(const float16_t& lo, const float16_t& hi, float s) {
  u32x6_t r;
  asm("v_cvt_scalef32_2xpk16_fp6_f32 %0, %1, %2, %3" : "=&v"(r) : "v"(lo), "v"(hi), "v"(s));
  return r;
}
__device__ inline float32_t from_fp6x32(const u32x6_t& v, float s) {
  float32_t r;
  asm("v_cvt_scalef32_pk32_f32_fp6 %0, %1, %2" : "=&v"(r) : "v"(v), "v"(s));
  return r;
}

// v: a block's 32 activations in fp32.
__device__ inline MxPieces mx_split(const float (&v)[kMxBlock]) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kMxBlock; ++i) amax = mx_absmax(amax, v[i]);
  const uint32_t bits = __builtin_bit_cast(uint32_t, amax);
  const uint32_t e = bits >> 23;
  MxPieces r;
  // exponent less 2, one more where the significand exceeds 7.5 / 4
  int b = (int)e - 2 + ((bits & 0x007FFFFFu) > 0x00700000u ? 1 : 0);
  const bool finite = e != 255u;
  b = b < kMxMinSplit ? kMxMinSplit : b;
  if (!finite) b = 127;
  float16_t lo, hi;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    lo[i] = finite ? v[2 * i] : 0.0f;
    hi[i] = finite ? v[2 * i + 1] : 0.0f;
  }
#pragma unroll
  for (int p = 0; p < kMxPieces; ++p) {
    const float s = __builtin_bit_cast(float, (uint32_t)(b - kMxPieceShift[p]) << 23);
    r.p[p] = to_fp6x32(lo, hi, s);
    if (p + 1 < kMxPieces) {
      const float32_t back = from_fp6x32(r.p[p], s);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        lo[i] -= back[2 * i];
        hi[i] -= back[2 * i + 1];
      }
    }
  }
  r.scale = finite ? (uint32_t)b | (uint32_t)(b - kMxPieceShift[1]) << 8 | (uint32_t)(b - kMxPieceShift[2]) << 16
                   : 0x00FFFFFFu;
  return r;
}

// Fragment-major storage of split activations.  A fragment is R rows (32 or
// 16) by 2048 / R elements of K (2 or 4 blocks): lane l of a wave holds row
// l % R, block l / R.  Per fragment and piece 64 lanes x 16 bytes, then 64
// lanes x 8 bytes; the scales are one dword per lane.  Fragments lie
// [row group][K step], rows past M and blocks past K are zeros.  With R = 16
// four steps make a super-step of 16 blocks, and lane group l / 16 holds block
// 4 (l / 16) + s of it at its step s.
constexpr int kMxPieceBytes = 64 * 24;
constexpr int kMxFragBytes = kMxPieces * kMxPieceBytes;
constexpr int kMxFragScaleBytes = 64 * 4;

template <class XT>
__device__ inline void mx_load_block(const uint16_t* __restrict__ p, float (&v)[kMxBlock]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const u32x4_t w = reinterpret_cast<const u32x4_t*>(p)[q];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[8 * q + 2 * e] = XT::to_f32((uint16_t)(w[e] & 0xFFFFu));
      v[8 * q + 2 * e + 1] = XT::to_f32((uint16_t)(w[e] >> 16));
    }
  }
}

__device__ inline void mx_store_pieces(const MxPieces& s, uint8_t* __restrict__ frag, uint32_t* __restrict__ fscale,
                                       int lane) {
#pragma unroll
  for (int p = 0; p < kMxPieces; ++p) {
    uint8_t* const q = frag + p * kMxPieceBytes;
    *reinterpret_cast<u32x4_t*>(q + 16 * lane) = u32x4_t{s.p[p][0], s.p[p][1], s.p[p][2], s.p[p][3]};
    *reinterpret_cast<u32x2_t*>(q + 1024 + 8 * lane) = u32x2_t{s.p[p][4], s.p[p][5]};
  }
  fscale[lane] = s.scale;
}

// Scale bytes 16 g .. 16 g + 15 of a row of nblk, 0 past its end (whatever codes
// stand there, times 2^-254 they are below fp32's smallest number), in each dword in
// the order 0, 2, 1, 3.
__device__ inline u32x4_t mx_scale_chunk(const uint8_t* __restrict__ row, int g, int nblk) {
  u32x4_t v = {0u, 0u, 0u, 0u};
  const uint8_t* const p = row + 16 * g;
  if (16 * g + 16 <= nblk) {
    __builtin_memcpy(&v, p, 16);
  } else {
#pragma unroll
    for (int q = 0; q < 16; ++q)
      if (16 * g + q < nblk) v[q / 4] |= (uint32_t)p[q] << (8 * (q % 4));
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = __builtin_amdgcn_perm(v[q], v[q], 0x03010200u);
  return v;
}

}  // namespace woq
