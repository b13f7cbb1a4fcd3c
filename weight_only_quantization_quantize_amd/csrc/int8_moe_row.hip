// The layer of experts (int8_moe.hip) for one token, in two launches, bound by streaming the
// chosen experts' weights once:
//   up    a workgroup quantizes the token's row for itself and takes columns of h: a gate and
//         an up row of a choice each time (two rows in flight for every sum)
//   down  a workgroup quantizes h's rows for itself, a wave holds up to CH pieces of 1024
//         elements of them, and takes columns of y: a row of every choice's expert
// The results are the tile path's to the last bit: exact sums, the same fp32 steps.
// bf16, H = 4096, I = 2048, 4 of 32 experts (101 MB): 23 .. 25 us (up 13 .. 15, 67 MB; down
// 9, 34 MB); the five launches of the tile path 43 .. 44.
#include "int8_row.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kWaves = 8;
constexpr int kMaxChunks = 4;
constexpr int kMaxChoices = 16;
constexpr int kTargetGroups = 512;

// H = 16 chunks, segs waves a row, CH chunks of 16 a lane.  h [top_k][I]; a choice of no
// expert here writes nothing.
template <class XT, int CH>
__global__ __launch_bounds__(kWaves * 64) void int8_moe_row_up_kernel(const void* __restrict__ x,
                                                                      const int32_t* __restrict__ experts,
                                                                      const int8_t* __restrict__ w, const float* __restrict__ sw,
                                                                      int chunks, int segs, int I, int E, int top_k,
                                                                      float* __restrict__ h) {
  constexpr int kPairs = 4 / CH;
  __shared__ int part[2][kPairs][2][kWaves];
  __shared__ uint32_t tops[kWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int seg = wave % segs, slot = wave / segs, slots = (int)(blockDim.x >> 6) / segs;
  const int K = chunks * 16, columns = top_k * I, stride = (int)gridDim.x * slots;
  int at[CH];
  bool live[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int chunk = (j * segs + seg) * 64 + lane;
    live[j] = chunk < chunks;
    at[j] = 16 * (live[j] ? chunk : chunks - 1);
  }
  auto expert = [&](int c) {  // clamped: loads stay inside the weights
    const int e = experts[c];
    return e < 0 ? 0 : (e < E ? e : E - 1);
  };
  u32x4_t c[2][kPairs][2][CH];
  auto load = [&](u32x4_t(&to)[kPairs][2][CH], int first) {
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      const int col = first + p * stride < columns ? first + p * stride : columns - 1;
      const int8_t* const row = w + ((int64_t)expert(col / I) * 2 * I + col % I) * K;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        to[p][0][j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(row + at[j]));
        to[p][1][j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(row + (int64_t)I * K + at[j]));
      }
    }
  };
  int first = (int)blockIdx.x * slots + slot;
  Int8RowLoad<CH> in;
  in.start(x, nullptr, at);
  __builtin_amdgcn_sched_barrier(0);
  load(c[0], first);
  __builtin_amdgcn_sched_barrier(0);
  uint32_t q[CH][4];
  const float scale = in.template codes<XT>(q, false, live, tops);
  const int batches = (columns + stride * kPairs - 1) / (stride * kPairs);
  auto batch = [&](int b, const u32x4_t(&from)[kPairs][2][CH]) {
#pragma unroll
    for (int p = 0; p < kPairs; ++p)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        int d = 0;
#pragma unroll
        for (int j = 0; j < CH; ++j) d = int8_dot16(from[p][s][j], q[j], d);
        d = wave_sum_last(d);
        if (lane == 63) part[b & 1][p][s][wave] = d;
      }
    __syncthreads();
    if ((int)threadIdx.x < kPairs * slots) {
      const int p = (int)threadIdx.x / slots, sl = (int)threadIdx.x % slots;
      const int col = (int)blockIdx.x * slots + sl + (b * kPairs + p) * stride;
      int g = 0, u = 0;
      for (int s = 0; s < segs; ++s) g += part[b & 1][p][0][sl * segs + s], u += part[b & 1][p][1][sl * segs + s];
      if (col < columns) {
        const int e = experts[col / I];
        if (e >= 0 && e < E) {
          const float* const s = sw + (int64_t)e * 2 * I + col % I;
          h[col] = int8_gated((float)g * scale * s[0], (float)u * scale * s[I]);
        }
      }
    }
    first += kPairs * stride;
  };
  for (int b = 0; b < batches; b += 2) {
    if (b + 1 < batches) load(c[1], first + kPairs * stride);
    batch(b, c[0]);
    if (b + 1 >= batches) break;
    if (b + 2 < batches) load(c[0], first + kPairs * stride);
    batch(b + 1, c[1]);
  }
}

// I = 16 chunks, segs pieces a choice; wave w holds the pieces w, w + 8, ...
template <class YT, int CH>
__global__ __launch_bounds__(kWaves * 64) void int8_moe_row_down_kernel(
    const float* __restrict__ h, const int32_t* __restrict__ experts, const float* __restrict__ weights,
    const int8_t* __restrict__ w, const float* __restrict__ sw, int chunks, int segs, int H, int E, int top_k,
    uint16_t* __restrict__ y) {
  constexpr int kSteps = 8 / CH;
  __shared__ int part[2][kSteps][kMaxChunks * kWaves];
  __shared__ uint32_t tops[kMaxChunks * kWaves];
  __shared__ float scales[kMaxChoices];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int I = chunks * 16, pieces = top_k * segs;
  auto is_here = [&](int e) { return e >= 0 && e < E; };
  int at[CH];
  const int8_t* row[CH];  // of y's column 0
  bool live[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int piece = wave + kWaves * j, of = piece < pieces ? piece / segs : 0, chunk = piece % segs * 64 + lane;
    const int e = experts[of];
    live[j] = piece < pieces && chunk < chunks && is_here(e);
    at[j] = 16 * (chunk < chunks ? chunk : chunks - 1);
    row[j] = w + (int64_t)(is_here(e) ? e : 0) * H * I + at[j];
    at[j] += of * I;
  }
  u32x4_t c[2][kSteps][CH];
  const int stride = (int)gridDim.x;
  auto load = [&](u32x4_t(&to)[kSteps][CH], int first) {
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      const int n = first + st * stride < H ? first + st * stride : H - 1;
#pragma unroll
      for (int j = 0; j < CH; ++j)
        to[st][j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(row[j] + (int64_t)n * I));
    }
  };
  int first = blockIdx.x;
  float f[CH][16];
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4_t v = *reinterpret_cast<const float4_t*>(h + at[j] + 4 * e);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[j][4 * e + i] = v[i];
    }
  __builtin_amdgcn_sched_barrier(0);
  load(c[0], first);
  __builtin_amdgcn_sched_barrier(0);
  uint32_t q[CH][4];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t b = magnitude(f[j][e]);
      top = top > b ? top : b;
    }
    top = wave_max_bits(top);
    if (lane == 0) tops[wave + kWaves * j] = top;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int of = wave + kWaves * j < pieces ? (wave + kWaves * j) / segs : 0;
    uint32_t top = 0;
    for (int s = 0; s < segs; ++s) {
      const uint32_t o = tops[of * segs + s];
      top = top > o ? top : o;
    }
    const Int8Row p = int8_row(top);
    int8_codes(f[j], p, q[j]);
#pragma unroll
    for (int e = 0; e < 4; ++e) q[j][e] = live[j] ? q[j][e] : 0u;
    if (lane == 0 && wave + kWaves * j < pieces && (wave + kWaves * j) % segs == 0) scales[of] = p.scale;
  }
  const int batches = (H + stride * kSteps - 1) / (stride * kSteps);
  auto batch = [&](int b, const u32x4_t(&from)[kSteps][CH]) {
    // thread (step, choice) of the sums below; its scale is on its way meanwhile
    const int st = (int)threadIdx.x / kMaxChoices, of = (int)threadIdx.x % kMaxChoices;
    const int n = (int)blockIdx.x + (b * kSteps + st) * stride;
    const bool sums = st < kSteps && of < top_k && n < H && is_here(experts[of < top_k ? of : 0]);
    const float s = sums ? sw[(int64_t)experts[of] * H + n] : 0.0f, weight = sums ? weights[of] : 0.0f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int d = wave_sum_last(int8_dot16(from[i][j], q[j], 0));
        if (lane == 63) part[b & 1][i][wave + kWaves * j] = d;
      }
    __syncthreads();
    if (wave < (kSteps * kMaxChoices + 63) / 64) {
      float p = 0.0f;
      if (sums) {
        int d = 0;
        for (int g = 0; g < segs; ++g) d += part[b & 1][st][of * segs + g];
        p = (float)d * scales[of] * s;
      }
      float v = 0.0f;  // in the order of choice; one of no expert here is left out
      for (int k = 0; k < top_k; ++k) {
        const int from_lane = (lane & ~(kMaxChoices - 1)) + k;
        const float a = __shfl(weight, from_lane, 64), o = __shfl(p, from_lane, 64);
        v = __shfl(sums ? 1 : 0, from_lane, 64) ? fmaf(a, o, v) : v;
      }
      if (of == 0 && st < kSteps && n < H) y[n] = YT::from_f32(v);
    }
    first += kSteps * stride;
  };
  for (int b = 0; b < batches; b += 2) {
    if (b + 1 < batches) load(c[1], first + kSteps * stride);
    batch(b, c[0]);
    if (b + 1 >= batches) break;
    if (b + 2 < batches) load(c[0], first + kSteps * stride);
    batch(b + 1, c[1]);
  }
}

int pieces(int64_t K) { return (int)((K / 16 + 63) / 64); }
int lane_chunks(int64_t pieces) { return pieces <= kWaves ? 1 : (pieces <= 2 * kWaves ? 2 : 4); }

template <class XT>
hipError_t launch(const void* X, const int32_t* experts, const float* weights, const int8_t* up, const float* up_scales,
                  const int8_t* down, const float* down_scales, int H, int I, int E, int top_k, uint16_t* Y, float* h,
                  hipStream_t stream) {
  const int ch = lane_chunks(pieces(H)), segs = (pieces(H) + ch - 1) / ch, slots = kWaves / segs;
  const int64_t columns = ((int64_t)top_k * I + slots - 1) / slots;
  auto* const f = ch == 1 ? int8_moe_row_up_kernel<XT, 1> : (ch == 2 ? int8_moe_row_up_kernel<XT, 2> : int8_moe_row_up_kernel<XT, 4>);
  f<<<(unsigned)(columns < kTargetGroups ? columns : kTargetGroups), (unsigned)(slots * segs * 64), 0, stream>>>(
      X, experts, up, up_scales, H / 16, segs, I, E, top_k, h);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int ph = pieces(I), chd = lane_chunks((int64_t)ph * top_k);
  auto* const g = chd == 1 ? int8_moe_row_down_kernel<XT, 1> : (chd == 2 ? int8_moe_row_down_kernel<XT, 2> : int8_moe_row_down_kernel<XT, 4>);
  g<<<(unsigned)(H < kTargetGroups ? H : kTargetGroups), kWaves * 64, 0, stream>>>(h, experts, weights, down, down_scales, I / 16, ph, H,
                                                                                  E, top_k, Y);
  return hipGetLastError();
}

}  // namespace

bool int8_moe_row_supported(int64_t H, int64_t I, int64_t top_k) {
  return top_k <= kMaxChoices && pieces(H) <= kMaxChunks * kWaves && pieces(I) * top_k <= kMaxChunks * kWaves;
}

hipError_t launch_int8_moe_row(const void* X, int xdtype, const int32_t* experts, const float* weights, const void* up,
                               const float* up_scales, const void* down, const float* down_scales, int64_t H, int64_t I, int64_t E,
                               int top_k, void* Y, void* workspace, hipStream_t stream) {
  auto* const f = xdtype == 0 ? launch<F16> : launch<BF16>;
  return f(X, experts, weights, static_cast<const int8_t*>(up), up_scales, static_cast<const int8_t*>(down), down_scales, (int)H,
           (int)I, (int)E, top_k, static_cast<uint16_t*>(Y), static_cast<float*>(workspace), stream);
}

}  // namespace woq
