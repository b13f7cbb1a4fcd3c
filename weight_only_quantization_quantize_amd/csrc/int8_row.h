// What the kernels that stream weights past one row share (int8_gemv.hip, int8_moe_row.hip).
#pragma once

#include "int8_device.h"

namespace woq {

// The sum over a wave, in lane 63.
__device__ inline int wave_sum_last(int v) {
  auto step = [&](auto ctrl, auto rows) {
    v += __builtin_amdgcn_update_dpp(0, v, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
  };
  step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xF>{});  // row_shr 1, 2, 4, 8
  step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});  // row_bcast 15, 31
  step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});
  return v;
}

// A lane's 16 CH elements of a row of 16-bit x (at: where each 16 begin; inside the row), on
// their way, with the channels' scales where there are some.
template <int CH>
struct Int8RowLoad {
  u32x4_t v[CH][2];
  float4_t s[CH][4];
  __device__ __forceinline__ void start(const void* __restrict__ x, const float* __restrict__ act_scale, const int (&at)[CH]) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const u32x4_t* const p = reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(x) + at[j]);
      v[j][0] = p[0], v[j][1] = p[1];
      if (act_scale)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = *reinterpret_cast<const float4_t*>(act_scale + at[j] + 4 * e);
    }
  }
  // The codes, 0 where live says no, and the row's scale; the lanes of the workgroup hold all
  // of the row (some of it twice).  tops: LDS, a word for each wave.
  template <class XT>
  __device__ __forceinline__ float codes(uint32_t (&q)[CH][4], bool scaled, const bool (&live)[CH], uint32_t* tops) const {
    float f[CH][16];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) f[j][e] = XT::to_f32((uint16_t)(v[j][e / 8][e % 8 / 2] >> (16 * (e % 2))));
    if (scaled)
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) f[j][e] /= s[j][e / 4][e % 4];
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t b = magnitude(f[j][e]);
        top = top > b ? top : b;
      }
    top = wave_max_bits(top);
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    for (int i = 0; i < (int)(blockDim.x >> 6); ++i) {
      const uint32_t o = tops[i];
      top = top > o ? top : o;
    }
    const Int8Row p = int8_row(top);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      int8_codes(f[j], p, q[j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) q[j][e] = live[j] ? q[j][e] : 0u;
    }
    return p.scale;
  }
};

__device__ inline int int8_dot16(u32x4_t w, const uint32_t (&q)[4], int sum) {
#pragma unroll
  for (int e = 0; e < 4; ++e) sum = __builtin_amdgcn_sdot4((int)w[e], (int)q[e], sum, false);
  return sum;
}

}  // namespace woq
