// A few rows of activations (MR: 1, 2 or 4; the last ones may be there twice) by 8-bit
// integer weights:
//   y[m, n] = (acc sa[m]) sw[n] + bias[n],  acc = sum_k q[m, k] w[n, k]
// for given codes q, or for 16-bit x that is quantized by every workgroup for itself: a lane
// needs the codes of the very 16 elements that it quantizes, and all that passes between
// lanes is the largest magnitude.
//
// Bound by streaming the weights once: 8192 x 8192 14 .. 15 us (4.7 TB/s) with the
// quantization in it, 19.5 with a launch before for the codes.
//
// A lane owns 16 k (CH times), 16 bytes of a row; a row's chunks are spread over `team` lanes
// (a power of two up to 64; longer rows over `segs` waves, the slots of a workgroup being
// 8 / segs rows).  Workgroup b takes the row groups b, b + B, ..., so the whole GPU reads one
// window of rows at a time, kSteps of them a batch, the next batch on its way while one is
// multiplied (v_dot4) and summed.
#include "int8_row.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kWaves = 8;
constexpr int kMaxChunks = 4;   // a lane's
constexpr int kTargetGroups = 512;

struct Codes {};  // of the row: given

template <class XT, class YT, int CH, int MR>
__global__ __launch_bounds__(kWaves * 64) void int8_gemv_kernel(const void* __restrict__ x, const float* __restrict__ sa,
                                                                const float* __restrict__ act_scale,
                                                                const int8_t* __restrict__ w, const float* __restrict__ sw,
                                                                const float* __restrict__ bias, int M, int N, int chunks, int segs,
                                                                int team, typename Int8Out<YT>::type* __restrict__ y) {
  constexpr int kSteps = MR == 4 ? 4 : 8 / CH;
  constexpr bool kGiven = std::is_same_v<XT, Codes>;
  __shared__ int part[2][kSteps][MR][kWaves];
  __shared__ uint32_t tops[MR][kWaves];
  __shared__ float scales[MR];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int seg = wave % segs, slot = wave / segs, waves = (int)(blockDim.x >> 6), slots = waves / segs;
  const int rpw = 64 / team, rows = slots * rpw;  // of a wave, of a workgroup's step
  const int K = chunks * 16;
  int chunk[CH], at[CH];  // the lane's; clamped: loads stay inside the row
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    chunk[j] = (j * segs + seg) * 64 + lane % team;
    at[j] = 16 * (chunk[j] < chunks ? chunk[j] : chunks - 1);
  }
  const int stride = (int)gridDim.x * rows;
  int row = (int)blockIdx.x * rows + slot * rpw + lane / team;
  u32x4_t c[2][kSteps][CH];
  auto load = [&](u32x4_t(&to)[kSteps][CH], int r0) {
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      const int r = r0 + st * stride;
      const int8_t* const p = w + (int64_t)(r < N ? r : N - 1) * K;
#pragma unroll
      for (int j = 0; j < CH; ++j) to[st][j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p + at[j]));
    }
  };
  // the rows' codes, while the first weights come
  uint32_t q[MR][CH][4];
  float scale[MR];
  bool live[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) live[j] = chunk[j] < chunks;
  auto of = [&](int m) { return (int64_t)(m < M ? m : M - 1); };
  if constexpr (kGiven) {
#pragma unroll
    for (int m = 0; m < MR; ++m) {
      scale[m] = sa[of(m)];
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(static_cast<const int8_t*>(x) + of(m) * K + at[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) q[m][j][e] = live[j] ? v[e] : 0u;
      }
    }
    load(c[0], row);
  } else {
    Int8RowLoad<CH> in[MR];
#pragma unroll
    for (int m = 0; m < MR; ++m) in[m].start(static_cast<const uint16_t*>(x) + of(m) * K, act_scale, at);
    __builtin_amdgcn_sched_barrier(0);
    load(c[0], row);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < MR; ++m) scale[m] = in[m].template codes<XT>(q[m], act_scale != nullptr, live, tops[m]);
  }
  if (threadIdx.x == 0)  // before the first batch's barrier
#pragma unroll
    for (int m = 0; m < MR; ++m) scales[m] = scale[m];
  auto store = [&](int m, int n, int sum, float by) {
    const float v = fmaf((float)sum * by, sw[n], bias ? bias[n] : 0.0f);  // as the tiles do (int8_gemm.hip)
    if (m < M) y[(int64_t)m * N + n] = Int8Out<YT>::of(v);
  };
  const int batches = (N + stride * kSteps - 1) / (stride * kSteps);
  auto batch = [&](int b, const u32x4_t(&from)[kSteps][CH]) {
    int sum[kSteps][MR];
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
#pragma unroll
      for (int m = 0; m < MR; ++m) {
        int d = 0;
#pragma unroll
        for (int j = 0; j < CH; ++j) d = int8_dot16(from[st][j], q[m][j], d);
        sum[st][m] = d;
      }
    if (segs == 1) {  // a row inside a wave
      if (team == 64) {
#pragma unroll
        for (int st = 0; st < kSteps; ++st)
#pragma unroll
          for (int m = 0; m < MR; ++m) sum[st][m] = wave_sum_last(sum[st][m]);
      } else {
        for (int off = team >> 1; off > 0; off >>= 1)
#pragma unroll
          for (int st = 0; st < kSteps; ++st)
#pragma unroll
            for (int m = 0; m < MR; ++m) sum[st][m] += __shfl_xor(sum[st][m], off, 64);
      }
      if (lane % team == team - 1)
#pragma unroll
        for (int st = 0; st < kSteps; ++st)
#pragma unroll
          for (int m = 0; m < MR; ++m)
            if (row + st * stride < N) store(m, row + st * stride, sum[st][m], scale[m]);
    } else {
#pragma unroll
      for (int st = 0; st < kSteps; ++st)
#pragma unroll
        for (int m = 0; m < MR; ++m) {
          const int d = wave_sum_last(sum[st][m]);
          if (lane == 63) part[b & 1][st][m][wave] = d;
        }
      __syncthreads();
      if ((int)threadIdx.x < kSteps * MR * slots) {
        const int i = (int)threadIdx.x / slots, m = i % MR, st = i / MR, sl = (int)threadIdx.x % slots;
        const int n = (int)blockIdx.x * rows + sl + (b * kSteps + st) * stride;
        int d = 0;
        for (int g = 0; g < segs; ++g) d += part[b & 1][st][m][sl * segs + g];
        if (n < N) store(m, n, d, scales[m]);
      }
    }
    row += kSteps * stride;
  };
  for (int b = 0; b < batches; b += 2) {
    if (b + 1 < batches) load(c[1], row + kSteps * stride);
    batch(b, c[0]);
    if (b + 1 >= batches) break;
    if (b + 2 < batches) load(c[0], row + kSteps * stride);
    batch(b + 1, c[1]);
  }
}

template <class XT, class YT>
hipError_t launch(const void* x, const float* sa, const float* act_scale, const void* w, const float* sw, const float* bias,
                  int M, int N, int K, void* y, hipStream_t stream) {
  const int chunks = K / 16;
  int ch = 1;
  while (chunks > ch * 64 * kWaves) ch *= 2;
  const int segs = (chunks + ch * 64 - 1) / (ch * 64);
  int team = 64;
  if (segs == 1)
    while (team > 1 && team / 2 >= chunks) team /= 2;
  const int slots = kWaves / segs, rows = slots * (64 / team);
  const int groups = (N + rows - 1) / rows;
  const unsigned grid = (unsigned)(groups < kTargetGroups ? groups : kTargetGroups);
  auto* const f = [&] {
    if constexpr (std::is_same_v<XT, Codes>)
      if (M > 2) return int8_gemv_kernel<XT, YT, 1, 4>;
    if (M == 2) return int8_gemv_kernel<XT, YT, 1, 2>;
    return ch == 1 ? int8_gemv_kernel<XT, YT, 1, 1> : (ch == 2 ? int8_gemv_kernel<XT, YT, 2, 1> : int8_gemv_kernel<XT, YT, kMaxChunks, 1>);
  }();
  f<<<grid, (unsigned)(slots * segs * 64), 0, stream>>>(x, sa, act_scale, static_cast<const int8_t*>(w), sw, bias, M, N, chunks, segs,
                                                        team, static_cast<typename Int8Out<YT>::type*>(y));
  return hipGetLastError();
}

}  // namespace

// More rows of longer ones would not leave the registers for the weights on their way, and
// so would quantizing more than two: 8192 x 8192 takes 14.5, 16, 17, 17 us for 1 .. 4 rows of
// codes (32 x 32 tiles: 18), 14.7 and 16 for 1 and 2 of 16-bit activations, 31 for 3 and 4 (with
// a launch before for the codes 20).
int64_t int8_gemv_max_rows(int64_t K) { return K <= kWaves * 64 * 16 ? 4 : (K <= kMaxChunks * kWaves * 64 * 16 ? 1 : 0); }
int64_t int8_linear_max_rows(int64_t K) {
  const int64_t n = int8_gemv_max_rows(K);
  return n < 2 ? n : 2;
}

hipError_t launch_int8_gemv(const void* codes, const float* a_scales, const void* W, const float* w_scales, const float* bias,
                            int64_t M, int64_t N, int64_t K, int ydtype, void* y, hipStream_t stream) {
  auto* const f = ydtype == 0 ? launch<Codes, F16> : (ydtype == 1 ? launch<Codes, BF16> : launch<Codes, F32>);
  return f(codes, a_scales, nullptr, W, w_scales, bias, (int)M, (int)N, (int)K, y, stream);
}

hipError_t launch_int8_linear_rows(const void* x, int xdtype, const float* act_scale, const void* W, const float* w_scales,
                                   const float* bias, int64_t M, int64_t N, int64_t K, void* y, hipStream_t stream) {
  auto* const f = xdtype == 0 ? launch<F16, F16> : launch<BF16, BF16>;
  return f(x, nullptr, act_scale, W, w_scales, bias, (int)M, (int)N, (int)K, y, stream);
}

}  // namespace woq
