// One row of activations by 8-bit integer weights:
//   y[n] = (acc sa) sw[n] + bias[n],  acc = sum_k q[k] w[n, k]
// for given codes q, or for 16-bit x that is quantized by every workgroup for itself: a lane
// needs the codes of the very 16 elements that it quantizes, and all that passes between
// lanes is the largest magnitude.
//
// Bound by streaming the weights once.  A lane owns 16 k (CH times), 16 bytes of a row; a
// row's chunks are spread over `team` lanes (a power of two up to 64; longer rows over
// `segs` waves, the slots of a workgroup being 8 / segs rows).  Workgroup b takes the row
// groups b, b + B, ..., so the whole GPU reads one window of rows at a time, kSteps of them
// a batch, the next batch on its way while one is multiplied (v_dot4) and summed.
#include "int8_row.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kWaves = 8;
constexpr int kMaxChunks = 4;   // a lane's
constexpr int kTargetGroups = 512;

struct Codes {};  // of the row: given

template <class XT, class YT, int CH>
__global__ __launch_bounds__(kWaves * 64) void int8_gemv_kernel(const void* __restrict__ x, const float* __restrict__ sa,
                                                                const float* __restrict__ act_scale,
                                                                const int8_t* __restrict__ w, const float* __restrict__ sw,
                                                                const float* __restrict__ bias, int N, int chunks, int segs,
                                                                int team, typename Int8Out<YT>::type* __restrict__ y) {
  constexpr int kSteps = CH == 1 ? 8 : 8 / CH;
  constexpr bool kGiven = std::is_same_v<XT, Codes>;
  __shared__ int part[2][kSteps][kWaves];
  __shared__ uint32_t tops[kWaves];
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
  // the row's codes, while the first weights come
  uint32_t q[CH][4];
  float scale;
  if constexpr (kGiven) {
    u32x4_t v[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) v[j] = *reinterpret_cast<const u32x4_t*>(static_cast<const int8_t*>(x) + at[j]);
    scale = sa[0];
    load(c[0], row);
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) q[j][e] = chunk[j] < chunks ? v[j][e] : 0u;
  } else {
    Int8RowLoad<CH> in;
    in.start(x, act_scale, at);
    __builtin_amdgcn_sched_barrier(0);
    load(c[0], row);
    __builtin_amdgcn_sched_barrier(0);
    bool live[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) live[j] = chunk[j] < chunks;
    scale = in.template codes<XT>(q, act_scale != nullptr, live, tops);
  }
  auto store = [&](int n, int sum) {
    float v = (float)sum * scale * sw[n];
    if (bias) v += bias[n];
    y[n] = Int8Out<YT>::of(v);
  };
  const int batches = (N + stride * kSteps - 1) / (stride * kSteps);
  auto batch = [&](int b, const u32x4_t(&from)[kSteps][CH]) {
    int sum[kSteps];
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      int d = 0;
#pragma unroll
      for (int j = 0; j < CH; ++j) d = int8_dot16(from[st][j], q[j], d);
      sum[st] = d;
    }
    if (segs == 1) {  // a row inside a wave
      if (team == 64) {
#pragma unroll
        for (int st = 0; st < kSteps; ++st) sum[st] = wave_sum_last(sum[st]);
      } else {
        for (int off = team >> 1; off > 0; off >>= 1)
#pragma unroll
          for (int st = 0; st < kSteps; ++st) sum[st] += __shfl_xor(sum[st], off, 64);
      }
#pragma unroll
      for (int st = 0; st < kSteps; ++st)
        if (lane % team == team - 1 && row + st * stride < N) store(row + st * stride, sum[st]);
    } else {
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const int d = wave_sum_last(sum[st]);
        if (lane == 63) part[b & 1][st][wave] = d;
      }
      __syncthreads();
      if ((int)threadIdx.x < kSteps * slots) {
        const int st = (int)threadIdx.x / slots, sl = (int)threadIdx.x % slots;
        const int n = (int)blockIdx.x * rows + sl + (b * kSteps + st) * stride;
        int d = 0;
        for (int g = 0; g < segs; ++g) d += part[b & 1][st][sl * segs + g];
        if (n < N) store(n, d);
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
                  int N, int K, void* y, hipStream_t stream) {
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
  auto* const f = ch == 1 ? int8_gemv_kernel<XT, YT, 1> : (ch == 2 ? int8_gemv_kernel<XT, YT, 2> : int8_gemv_kernel<XT, YT, kMaxChunks>);
  f<<<grid, (unsigned)(slots * segs * 64), 0, stream>>>(x, sa, act_scale, static_cast<const int8_t*>(w), sw, bias, N, chunks, segs,
                                                        team, static_cast<typename Int8Out<YT>::type*>(y));
  return hipGetLastError();
}

}  // namespace

int64_t int8_gemv_max_k() { return (int64_t)kMaxChunks * kWaves * 64 * 16; }

hipError_t launch_int8_gemv(const void* codes, const float* a_scales, const void* W, const float* w_scales, const float* bias,
                            int64_t N, int64_t K, int ydtype, void* y, hipStream_t stream) {
  auto* const f = ydtype == 0 ? launch<Codes, F16> : (ydtype == 1 ? launch<Codes, BF16> : launch<Codes, F32>);
  return f(codes, a_scales, nullptr, W, w_scales, bias, (int)N, (int)K, y, stream);
}

hipError_t launch_int8_linear_row(const void* x, int xdtype, const float* act_scale, const void* W, const float* w_scales,
                                  const float* bias, int64_t N, int64_t K, void* y, hipStream_t stream) {
  auto* const f = xdtype == 0 ? launch<F16, F16> : launch<BF16, BF16>;
  return f(x, nullptr, act_scale, W, w_scales, bias, (int)N, (int)K, y, stream);
}

}  // namespace woq
