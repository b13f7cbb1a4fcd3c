// Rows to codes and scales (int8_device.h), W waves a row; int8_quantize.hip has the kernel.
#pragma once

#include "int8_device.h"

namespace woq {

constexpr int kLaneElements = 8;
constexpr int kStepElements = 64 * kLaneElements;  // of a wave
constexpr int kRowMaxWaves = 16;

enum Fold { kNone, kMultiply, kDivide };

template <class XT>
struct Raw {
  u32x4_t v[kElementBytes<XT> / 2];
};

template <class XT>
__device__ inline void load_raw(Raw<XT>& raw, const void* __restrict__ row, int k) {
  const uint8_t* const p = static_cast<const uint8_t*>(row) + (int64_t)k * kElementBytes<XT>;
#pragma unroll
  for (int i = 0; i < kElementBytes<XT> / 2; ++i) raw.v[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p) + i);
}

template <class XT, Fold F>
__device__ inline void widen(float (&y)[kLaneElements], const Raw<XT>& raw, const float* __restrict__ s, int k) {
#pragma unroll
  for (int i = 0; i < kLaneElements; ++i) {
    if constexpr (kElementBytes<XT> == 4) {
      y[i] = __builtin_bit_cast(float, (uint32_t)raw.v[i / 4][i % 4]);
    } else {
      y[i] = XT::to_f32((uint16_t)(raw.v[0][i / 2] >> (16 * (i % 2))));
    }
  }
  if constexpr (F != kNone) {
    const float4_t a = *reinterpret_cast<const float4_t*>(s + k), b = *reinterpret_cast<const float4_t*>(s + k + 4);
#pragma unroll
    for (int i = 0; i < kLaneElements; ++i) {
      const float c = i < 4 ? a[i % 4] : b[i % 4];
      y[i] = F == kMultiply ? y[i] * c : y[i] / c;
    }
  }
}

// The largest magnitude's bits so far.  16-bit elements as they come are compared in pairs
// (their bits are in the order of their magnitudes, infinity and NaN above all).
template <class XT, Fold F>
struct Largest {
  static constexpr bool kPairs = kElementBytes<XT> == 2 && F == kNone;
  typedef uint16_t pair_t __attribute__((ext_vector_type(2)));
  uint32_t top = 0;
  __device__ inline void take(const Raw<XT>& raw, const float (&y)[kLaneElements]) {
    if constexpr (kPairs) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        top = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(pair_t, top),
                                                                      __builtin_bit_cast(pair_t, (uint32_t)raw.v[0][i] & 0x7FFF7FFFu)));
    } else {
#pragma unroll
      for (int i = 0; i < kLaneElements; ++i) {
        const uint32_t b = magnitude(y[i]);
        top = top > b ? top : b;
      }
    }
  }
  __device__ inline uint32_t bits() const {
    if constexpr (kPairs) {
      const uint32_t a = top & 0xFFFFu, b = top >> 16;
      return magnitude(XT::to_f32((uint16_t)(a > b ? a : b)));
    }
    return top;
  }
};

// W waves a row, as many rows as they are times in a workgroup, the block-th of its kind.
// rounds: times STEPS steps of the row's waves cover the row; 1: it stays in registers.
template <class XT, Fold F, int STEPS>
__device__ __forceinline__ void int8_quantize_rows(const void* __restrict__ x, const float* __restrict__ s, int64_t M, int K, int W,
                                                   int rounds, int64_t block, int8_t* __restrict__ codes,
                                                   float* __restrict__ scales) {
  __shared__ uint32_t tops[kRowMaxWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rows = (int)(blockDim.x >> 6) / W, w = wave % W;
  const int64_t m = block * rows + wave / W;
  const bool live = m < M;
  const uint8_t* const row = static_cast<const uint8_t*>(x) + (live ? m : 0) * K * kElementBytes<XT>;
  Raw<XT> raw[STEPS];
  float y[STEPS][kLaneElements];
  Largest<XT, F> largest;
  auto at = [&](int round, int i) { return ((round * STEPS + i) * W + w) * kStepElements + kLaneElements * lane; };
  for (int round = 0; round < rounds; ++round) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
      if (at(round, i) < K) load_raw<XT>(raw[i], row, at(round, i));
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
      if (at(round, i) < K) {
        widen<XT, F>(y[i], raw[i], s, at(round, i));
        largest.take(raw[i], y[i]);
      }
  }
  uint32_t top = largest.bits();
  top = wave_max_bits(top);
  if (W > 1) {
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    for (int i = 0; i < W; ++i) {
      const uint32_t o = tops[wave - w + i];
      top = top > o ? top : o;
    }
  }
  if (!live) return;
  const Int8Row p = int8_row(top);
  if (w == 0 && lane == 0) scales[m] = p.scale;
  for (int round = 0; round < rounds; ++round) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
      if (at(round, i) < K) {
        if (rounds > 1) {
          load_raw<XT>(raw[i], row, at(round, i));
          widen<XT, F>(y[i], raw[i], s, at(round, i));
        }
        uint32_t q[2];
        int8_codes(y[i], p, q);
        *reinterpret_cast<u32x2_t*>(codes + m * K + at(round, i)) = u32x2_t{q[0], q[1]};
      }
  }
}

// How a matrix's rows are shared out: W, rounds and rows a workgroup.  A launch has fewer than
// 2^32 threads: workgroups of more rows than that go around (kMostGroups of up to 1024 threads).
constexpr unsigned kMostGroups = 1u << 21;
struct Int8RowsPlan {
  int W, per, rows;
  unsigned groups;
  int threads() const { return rows * W * 64; }
  int rounds() const { return (per + 3) / 4; }
};
inline Int8RowsPlan int8_rows_plan(int64_t M, int64_t K) {
  const int steps = (int)((K + kStepElements - 1) / kStepElements);  // of one wave
  Int8RowsPlan p;
  p.W = 1;
  while (p.W < kRowMaxWaves && (p.W * 4 < steps || (p.W < steps && M * p.W < 2048))) p.W *= 2;
  p.per = (steps + p.W - 1) / p.W;
  p.rows = p.W >= 4 ? 1 : 4 / p.W;
  p.groups = (unsigned)((M + p.rows - 1) / p.rows);
  return p;
}

}  // namespace woq
