// The inner loop of the products that stream microscaled weights past a few
// rows of activations: a wave multiplies NT tiles of 16 weight rows by TC
// chunks of 16 activation rows over its K steps of 128, on
// v_mfma_scale_f32_16x16x128_f8f6f4 with activations split into 6-bit pieces
// (mxfp4_device.h).
//
// Lane (r, q) (r = lane % 16, q = lane / 16) supplies block q of a K step for
// weight row r (16 bytes as stored, one scale byte) and for activation row r
// (a fragment's lane): the weights go from memory to the matrix unit without a
// decode or a turn through LDS.
#pragma once

#include "mxfp4_device.h"

namespace woq {

// One K step of a wave's weights.
template <int NT>
struct MxWeights {
  u32x4_t c[NT];
  uint32_t s[NT];
};

// codes / scales: lane's block of tile 0; tile j is tile_stride blocks further.
template <int NT>
__device__ inline void mx_load_weights(MxWeights<NT>& w, const uint8_t* __restrict__ codes,
                                       const uint8_t* __restrict__ scales, const int64_t (&tile)[NT]) {
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    w.c[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(codes + 16 * tile[j]));
    w.s[j] = scales[tile[j]];
  }
}

// One K step of one chunk's activations.
struct MxActivations {
  i32x8_t p0, p1, p2;
  int s;
};

__device__ inline void mx_load_activations(MxActivations& a, const uint8_t* __restrict__ frag,
                                           const uint32_t* __restrict__ fscale, int lane) {
  auto piece = [&](int p) {
    return mx_operand(*reinterpret_cast<const u32x4_t*>(frag + p * kMxPieceBytes + 16 * lane),
                      *reinterpret_cast<const u32x2_t*>(frag + p * kMxPieceBytes + 1024 + 8 * lane));
  };
  a.p0 = piece(0);
  a.p1 = piece(1);
  a.p2 = piece(2);
  a.s = (int)fscale[lane];
}

// acc += activations (rows of D) x weights (columns of D), smallest piece first.
template <int NT>
__device__ inline void mx_multiply(float4_t (&acc)[NT], const MxActivations& a, const MxWeights<NT>& w) {
#pragma unroll
  for (int j = 0; j < NT; ++j)
    acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.p2, mx_operand(w.c[j]), acc[j],
                                                              kMfmaFp6, kMfmaFp4, 2, a.s, 0, (int)w.s[j]);
#pragma unroll
  for (int j = 0; j < NT; ++j)
    acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.p1, mx_operand(w.c[j]), acc[j],
                                                              kMfmaFp6, kMfmaFp4, 1, a.s, 0, (int)w.s[j]);
#pragma unroll
  for (int j = 0; j < NT; ++j)
    acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.p0, mx_operand(w.c[j]), acc[j],
                                                              kMfmaFp6, kMfmaFp4, 0, a.s, 0, (int)w.s[j]);
}

}  // namespace woq
