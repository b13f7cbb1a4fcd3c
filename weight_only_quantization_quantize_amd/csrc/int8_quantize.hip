// Rows to 8-bit integers with a scale each (int8_device.h): y = x, x s or x / s of the
// channel scales s, rounded to fp32; scale = max|y| / 127; codes.
//
// Bound by reading x and writing the codes: 28672 x 8192 fp16 with folded scales 156 .. 162 us,
// 4.4 TB/s, where a copy makes 5.1 (192 us with the rounding's steps one by one; int8_device.h).
//
// A row stays in the registers of its W waves
// between the search for its largest magnitude and the rounding (8 elements a lane and
// step, up to 4 steps; longer rows are read a second time, out of L2).  One wave a
// row where there are rows for the whole GPU, up to 16 where there are few.
#include "int8_rows.h"
#include "woq_internal.h"

namespace woq {
namespace {

template <class XT, Fold F, int STEPS>
__global__ __launch_bounds__(kRowMaxWaves * 64) void int8_quantize_kernel(const void* __restrict__ x,
                                                                         const float* __restrict__ s, int64_t M, int K, int W,
                                                                         int rounds, unsigned groups, int8_t* __restrict__ codes,
                                                                         float* __restrict__ scales) {
  for (unsigned g = blockIdx.x; g < groups; g += gridDim.x) {
    int8_quantize_rows<XT, F, STEPS>(x, s, M, K, W, rounds, g, codes, scales);
    if (g + gridDim.x < groups) __syncthreads();  // the waves' largest magnitudes were read
  }
}

template <class XT, Fold F>
hipError_t launch(const void* x, const float* s, int64_t M, int K, void* codes, float* scales, hipStream_t stream) {
  const Int8RowsPlan p = int8_rows_plan(M, K);
  auto* const f = p.per <= 1 ? int8_quantize_kernel<XT, F, 1> : (p.per <= 2 ? int8_quantize_kernel<XT, F, 2> : int8_quantize_kernel<XT, F, 4>);
  const unsigned grid = p.groups < kMostGroups ? p.groups : kMostGroups;
  f<<<grid, (unsigned)p.threads(), 0, stream>>>(x, s, M, K, p.W, p.rounds(), p.groups, static_cast<int8_t*>(codes), scales);
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
