// Microscaled 4-bit floats (MXFP4): quantization, its inverse, and the split
// of 16-bit activations into the fragments that the products' kernels read.
//
// Quantization of a block of 32 values x (format in mxfp4_device.h):
//   b    = clamp(floor(log2 max|x|) - 2 + 127, 0, 254), 0 for a zero block
//   code = the e2m1 value nearest to x / 2^(b - 127), ties to the even code,
//          magnitudes above 6 to 6, the sign kept (a negative zero too)
// A block holding an infinity or a NaN gets b = 255 and zero codes.  gfx950's
// v_cvt_scalef32_pk_fp4_f32 does the scaling, rounding and saturation of two
// elements in one instruction.
//
// Bound by memory: 2 + 0.5 + 1/32 bytes per element, a dozen VALU operations.
// A lane takes 8 elements (one 16-byte load, one 4-byte store), four lanes a
// block, so that loads and stores of a wave are contiguous.
#include "mxfp4_device.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kThreads = 256;

// Codes of 8 elements with scale byte b.  The 16-bit forms of the conversion
// flush elements near the bottom of their type's range, so the elements go
// through fp32, and blocks of scales below 2^-63 (bf16 only) are raised by 2^64
// first, where no fp32 subnormal is left.  Both steps are exact.
template <class XT>
__device__ inline uint32_t to_fp4x8(u32x4_t w, uint32_t b) {
  const bool low = b < 64u;
  const float up = low ? 0x1p64f : 1.0f;
  const float s = mx_pow2(low ? b + 64u : b);
  float v[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = XT::to_f32((uint16_t)(w[e] & 0xFFFFu)) * up;
    v[2 * e + 1] = XT::to_f32((uint16_t)(w[e] >> 16)) * up;
  }
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  return c;
}

// units: 8-element pieces, a multiple of 4.
template <class XT>
__global__ __launch_bounds__(kThreads) void mxfp4_quantize_kernel(const u32x4_t* __restrict__ x, int64_t units,
                                                                  uint32_t* __restrict__ codes,
                                                                  uint8_t* __restrict__ scales) {
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < units; i += step) {
    const u32x4_t w = x[i];
    // the magnitudes of the 16-bit patterns order as the values do; a NaN is above infinity
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = w[e] & 0x7FFFu, hi = (w[e] >> 16) & 0x7FFFu;
      m = m > lo ? m : lo;
      m = m > hi ? m : hi;
    }
    uint32_t o = (uint32_t)__shfl_xor((int)m, 1, 64);
    m = m > o ? m : o;
    o = (uint32_t)__shfl_xor((int)m, 2, 64);
    m = m > o ? m : o;
    const uint32_t b = mx_scale_byte(XT::to_f32((uint16_t)m));
    const uint32_t c = to_fp4x8<XT>(w, b);
    codes[i] = b == (uint32_t)kMxNan ? 0u : c;
    if ((i & 3) == 0) scales[i >> 2] = (uint8_t)b;
  }
}

// out: 0 fp16, 1 bf16, 2 fp32.  The values are exact in bf16 and fp32 but for
// an overflow (6 2^127); fp16 rounds what lies outside its range.
template <int OUT>
__global__ __launch_bounds__(kThreads) void mxfp4_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                                    const uint8_t* __restrict__ scales, int64_t units,
                                                                    void* __restrict__ out) {
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < units; i += step) {
    const uint32_t c = codes[i], b = scales[i >> 2];
    const bool nan = b == (uint32_t)kMxNan;
    const float s = nan ? 1.0f : mx_pow2(b);
    if constexpr (OUT == 2) {
      float2_t v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1),
                       __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3)};
      const float n = __builtin_bit_cast(float, 0x7FC00000u);
      float4_t* const o = reinterpret_cast<float4_t*>(out) + 2 * i;
      o[0] = nan ? float4_t{n, n, n, n} : float4_t{v[0][0], v[0][1], v[1][0], v[1][1]};
      o[1] = nan ? float4_t{n, n, n, n} : float4_t{v[2][0], v[2][1], v[3][0], v[3][1]};
    } else {
      u32x4_t v;
      if constexpr (OUT == 0) {
        v = u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 0)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 1)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 2)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 3))};
      } else {
        v = u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3))};
      }
      const uint32_t n2 = OUT == 0 ? 0x7E007E00u : 0x7FC07FC0u;
      reinterpret_cast<u32x4_t*>(out)[i] = nan ? u32x4_t{n2, n2, n2, n2} : v;
    }
  }
}

// Scale bytes [rows, nblk] -> dwords [2 ceil(nblk / 8)][rows_pad], `past` in the place
// of rows and blocks that are not there.
constexpr int kScaleWaves = kThreads / 64;
static_assert(kMxScaleRowPad % 64 == 0, "a wave's rows are whole");
struct ScaleJob {
  const uint8_t* scales;
  uint32_t* out;
  int rows, rows_pad;
  uint32_t past;
};
// Workgroup `block` of a job's: 64 rows, each wave 16 blocks of them (a lane a row,
// so the writes are contiguous), the waves next to each other in the rows' lines.
__device__ inline void turn_scales(const ScaleJob& j, int nblk, int block) {
  const int ktiles = (nblk + 7) / 8 * 2, groups = j.rows_pad / 64;
  const int row = block % groups * 64 + ((int)threadIdx.x & 63), g = block / groups * kScaleWaves + ((int)threadIdx.x >> 6);
  if (4 * g >= ktiles) return;
  const uint32_t past = j.past * 0x01010101u;
  u32x4_t v = {past, past, past, past};
  if (row < j.rows) v = mx_scale_chunk(j.scales + (int64_t)row * nblk, g, nblk, j.past);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (4 * g + q < ktiles) j.out[(int64_t)(4 * g + q) * j.rows_pad + row] = v[q];
}

__global__ __launch_bounds__(kThreads) void mxfp4_scales_kernel(ScaleJob w, ScaleJob a, int nblk, int wblocks) {
  const bool first = (int)blockIdx.x < wblocks;
  turn_scales(first ? w : a, nblk, (int)blockIdx.x - (first ? 0 : wblocks));
}

// Workgroups [0, split) split X, the rest turn W's scales.
// One wave per fragment of R rows x 2048 / R elements (layout in
// mxfp4_device.h).
template <int R>
__global__ __launch_bounds__(kThreads) void mxfp4_split_kernel(const uint16_t* __restrict__ X, int M, int K,
                                                               int ksteps, int frags, uint8_t* __restrict__ out,
                                                               ScaleJob w, int split) {
  if ((int)blockIdx.x >= split) {
    turn_scales(w, K / kMxBlock, (int)blockIdx.x - split);
    return;
  }
  const int f = (int)blockIdx.x * (kThreads / 64) + (int)(threadIdx.x >> 6);
  if (f >= frags) return;
  const int lane = threadIdx.x & 63;
  const int row = (f / ksteps) * R + lane % R;
  const int ks = f % ksteps;
  const int blk = R == 32 ? 2 * ks + lane / 32 : 16 * (ks / 4) + 4 * (lane / 16) + ks % 4;
  const int k = blk * kMxBlock;
  u32x4_t v[4] = {};
  if (row < M && k < K)
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = reinterpret_cast<const u32x4_t*>(X + (int64_t)row * K + k)[j];
  uint8_t* const to = out + (int64_t)f * kMxFragBytes + 16 * lane;
#pragma unroll
  for (int j = 0; j < 4; ++j) *reinterpret_cast<u32x4_t*>(to + 1024 * j) = v[j];
}

// Workgroups of a scale job.
int64_t scale_blocks(int64_t rows, int64_t K) {
  return mxfp4_scale_rows(rows) / 64 * ((K + 512 * kScaleWaves - 1) / (512 * kScaleWaves));
}
ScaleJob scale_job(const void* scales, int64_t rows, void* out, uint32_t past) {
  return ScaleJob{static_cast<const uint8_t*>(scales), static_cast<uint32_t*>(out), (int)rows, (int)mxfp4_scale_rows(rows), past};
}

unsigned grid_for(int64_t units) {
  const int64_t b = (units + kThreads - 1) / kThreads;
  return (unsigned)(b < 16384 ? b : 16384);
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void* x, int xdtype, int64_t M, int64_t K, void* codes, void* scales,
                                 hipStream_t stream) {
  const int64_t units = M * K / 8;
  const auto* xp = static_cast<const u32x4_t*>(x);
  auto* cp = static_cast<uint32_t*>(codes);
  auto* sp = static_cast<uint8_t*>(scales);
  if (xdtype == 0)
    mxfp4_quantize_kernel<F16><<<grid_for(units), kThreads, 0, stream>>>(xp, units, cp, sp);
  else
    mxfp4_quantize_kernel<BF16><<<grid_for(units), kThreads, 0, stream>>>(xp, units, cp, sp);
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const void* codes, const void* scales, int64_t M, int64_t K, int outdtype,
                                   void* out, hipStream_t stream) {
  const int64_t units = M * K / 8;
  const auto* cp = static_cast<const uint32_t*>(codes);
  const auto* sp = static_cast<const uint8_t*>(scales);
  if (outdtype == 0)
    mxfp4_dequantize_kernel<0><<<grid_for(units), kThreads, 0, stream>>>(cp, sp, units, out);
  else if (outdtype == 1)
    mxfp4_dequantize_kernel<1><<<grid_for(units), kThreads, 0, stream>>>(cp, sp, units, out);
  else
    mxfp4_dequantize_kernel<2><<<grid_for(units), kThreads, 0, stream>>>(cp, sp, units, out);
  return hipGetLastError();
}

hipError_t launch_mxfp4_scales(const void* Ws, int64_t N, void* wout, const void* As, int64_t M, void* aout, int64_t K,
                               hipStream_t stream) {
  const int64_t wblocks = scale_blocks(N, K), ablocks = scale_blocks(M, K);
  mxfp4_scales_kernel<<<(unsigned)(wblocks + ablocks), kThreads, 0, stream>>>(
      scale_job(Ws, N, wout, 0u), scale_job(As, M, aout, 0u), (int)(K / kMxBlock), (int)wblocks);
  return hipGetLastError();
}

hipError_t launch_mxfp4_split(const void* X, int64_t M, int64_t K, int R, int64_t row_groups, int64_t ksteps, void* out,
                              const void* Ws, int64_t N, void* wout, hipStream_t stream) {
  const int frags = (int)(row_groups * ksteps);
  const int split = (frags + kThreads / 64 - 1) / (kThreads / 64);
  const unsigned grid = (unsigned)(split + (Ws ? scale_blocks(N, K) : 0));
  auto* const f = R == 32 ? mxfp4_split_kernel<32> : mxfp4_split_kernel<16>;
  f<<<grid, kThreads, 0, stream>>>(static_cast<const uint16_t*>(X), (int)M, (int)K, (int)ksteps, frags, static_cast<uint8_t*>(out),
                                   scale_job(Ws, N, wout, 127u), split);
  return hipGetLastError();
}

}  // namespace woq
