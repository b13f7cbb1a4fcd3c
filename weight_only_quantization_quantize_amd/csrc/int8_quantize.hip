// Rows to 8-bit integers with a scale each (int8_device.h): y = x, x s or x / s of the
// channel scales s, rounded to fp32; scale = max|y| / 127; codes.
//
// Bound by reading x and writing the codes.  A row stays in the registers of its W waves
// between the search for its largest magnitude and the rounding (8 elements a lane and
// step, up to kSteps steps; longer rows are read a second time, out of L2).  One wave a
// row where there are rows for the whole GPU, up to 16 where there are few.
#include "int8_device.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kLaneElements = 8;
constexpr int kStepElements = 64 * kLaneElements;  // of a wave
constexpr int kMaxWaves = 16;

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

// W waves a row, R rows a workgroup.  rounds: times STEPS steps of the row's waves
// cover the row; 1: it stays in registers.
template <class XT, Fold F, int STEPS>
__global__ __launch_bounds__(kMaxWaves * 64) void int8_quantize_kernel(const void* __restrict__ x,
                                                                      const float* __restrict__ s, int64_t M, int K,
                                                                      int W, int rounds, int8_t* __restrict__ codes,
                                                                      float* __restrict__ scales) {
  __shared__ uint32_t tops[kMaxWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rows = (int)(blockDim.x >> 6) / W, w = wave % W;
  const int64_t m = (int64_t)blockIdx.x * rows + wave / W;
  const bool live = m < M;
  const uint8_t* const row = static_cast<const uint8_t*>(x) + (live ? m : 0) * K * kElementBytes<XT>;
  Raw<XT> raw[STEPS];
  float y[kLaneElements];
  uint32_t top = 0;
  auto at = [&](int round, int i) { return ((round * STEPS + i) * W + w) * kStepElements + kLaneElements * lane; };
  for (int round = 0; round < rounds; ++round) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
      if (at(round, i) < K) load_raw<XT>(raw[i], row, at(round, i));
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
      if (at(round, i) < K) {
        widen<XT, F>(y, raw[i], s, at(round, i));
#pragma unroll
        for (int e = 0; e < kLaneElements; ++e) {
          const uint32_t b = magnitude(y[e]);
          top = top > b ? top : b;
        }
      }
  }
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
        if (rounds > 1) load_raw<XT>(raw[i], row, at(round, i));
        widen<XT, F>(y, raw[i], s, at(round, i));
        int8_codes(y, p);
        *reinterpret_cast<u32x2_t*>(codes + m * K + at(round, i)) =
            u32x2_t{int8_pack(y[0], y[1], y[2], y[3]), int8_pack(y[4], y[5], y[6], y[7])};
      }
  }
}

template <class XT, Fold F>
hipError_t launch(const void* x, const float* s, int64_t M, int K, void* codes, float* scales, hipStream_t stream) {
  const int steps = (K + kStepElements - 1) / kStepElements;  // of one wave
  int W = 1;
  while (W < kMaxWaves && (W * 4 < steps || (W < steps && M * W < 2048))) W *= 2;
  const int per = (steps + W - 1) / W;
  const int rows = W >= 4 ? 1 : 4 / W;
  const unsigned grid = (unsigned)((M + rows - 1) / rows);
  auto* const f = per <= 1 ? int8_quantize_kernel<XT, F, 1> : (per <= 2 ? int8_quantize_kernel<XT, F, 2> : int8_quantize_kernel<XT, F, 4>);
  f<<<grid, (unsigned)(rows * W * 64), 0, stream>>>(x, s, M, K, W, (per + 3) / 4, static_cast<int8_t*>(codes), scales);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_quantize(const void* x, int xdtype, const float* act_scale, bool multiply, int64_t M, int64_t K,
                                void* codes, float* scales, hipStream_t stream) {
  auto run = [&](auto tag) {
    using XT = decltype(tag);
    if (!act_scale) return launch<XT, kNone>(x, act_scale, M, (int)K, codes, scales, stream);
    return multiply ? launch<XT, kMultiply>(x, act_scale, M, (int)K, codes, scales, stream)
                    : launch<XT, kDivide>(x, act_scale, M, (int)K, codes, scales, stream);
  };
  return xdtype == 0 ? run(F16{}) : (xdtype == 1 ? run(BF16{}) : run(F32{}));
}

}  // namespace woq
