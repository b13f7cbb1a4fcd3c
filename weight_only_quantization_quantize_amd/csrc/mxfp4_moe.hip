// A mixture-of-experts layer on T <= 64 tokens with microscaled 4-bit experts:
//   logits[t, e] = sum_k x[t, k] router[e, k]                      (fp32)
//   S(t) = the top_k experts by (logit descending, index ascending)
//   p[t, e] = exp(logits[t, e]) / sum over S(t) of exp(logits)      for e in S(t)
//   h[t, e, i] = silu(x[t] . up[e, i]) (x[t] . up[e, I + i])        silu(g) = g / (1 + exp(-g))
//   y[t] = sum over S(t) of p[t, e] (down[e] h[t, e])               rounded once
//
// At a few tokens the layer is bound by streaming the chosen experts' weights
// (3 I H 17/32 bytes each) once, so each expert's weights are read once for all
// of its tokens: a tile of 16 weight rows meets all the tokens (chunks of 16)
// on the matrix units, where rows of tokens that did not choose the expert cost
// nothing that the stream does not hide, and no token is gathered.
//
// Three launches:
//   route  one workgroup per token: logits, choice, shares; x split into pieces
//   up     one workgroup per (expert, 32 columns of h): gate and up rows, then
//          p silu(g) u, split into pieces again (h keeps 14 bits of its block's
//          largest magnitude; the share is folded in here, where the values are
//          still fp32, so that the next product adds over experts by itself)
//   down   one workgroup per 16 columns of y, over all chosen experts: one
//          accumulator per token chunk takes every expert's products, in a
//          fixed order and without atomics.
#include <type_traits>

#include "mxfp4_stream.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kRouteThreads = 1024;
constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int kChunk = 16;
constexpr int kMaxTokens = 64;
constexpr int kMaxExperts = 512;
constexpr float kNotChosen = -1.0f;

// A logit's order as an unsigned number; a NaN comes below -infinity.
__device__ inline uint32_t order_key(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ inline uint64_t wave_max64(uint64_t v) {
  for (int off = 32; off > 0; off >>= 1) {
    const uint64_t o = ((uint64_t)(uint32_t)__shfl_xor((int)(v >> 32), off, 64) << 32) |
                       (uint32_t)__shfl_xor((int)(uint32_t)v, off, 64);
    v = v > o ? v : o;
  }
  return v;
}

// shares [E][64]: p[t, e], or kNotChosen (tokens past T too).
template <class XT>
__global__ __launch_bounds__(kRouteThreads) void moe_route_kernel(const uint16_t* __restrict__ X,
                                                                  const uint16_t* __restrict__ router, int T, int H,
                                                                  int E, int top_k, float* __restrict__ shares,
                                                                  uint8_t* __restrict__ xp, uint32_t* __restrict__ xs) {
  __shared__ float logit[kMaxExperts];
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ksteps = (H + 127) / 128;
  // split this token's row (rows of the last chunk past T: zeros)
  for (int b = threadIdx.x; b < 4 * ksteps; b += kRouteThreads) {
    float v[kMxBlock] = {};
    if (t < T && b * kMxBlock < H) mx_load_block<XT>(X + (int64_t)t * H + b * kMxBlock, v);
    const int64_t f = (int64_t)(t / kChunk) * ksteps + b / 4;
    mx_store_pieces(mx_split(v), xp + f * kMxFragBytes, xs + f * 64, (b % 4) * kChunk + t % kChunk);
  }
  if (t >= T) {
    for (int e = threadIdx.x; e < E; e += kRouteThreads) shares[e * kMaxTokens + t] = kNotChosen;
    return;
  }
  for (int e = wave; e < E; e += kRouteThreads / 64) {
    float a = 0.0f;
    for (int k = lane * 8; k < H; k += 512) {
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(X + (int64_t)t * H + k);
      const u32x4_t w = *reinterpret_cast<const u32x4_t*>(router + (int64_t)e * H + k);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a = fmaf(XT::to_f32((uint16_t)(v[j] & 0xFFFFu)), XT::to_f32((uint16_t)(w[j] & 0xFFFFu)), a);
        a = fmaf(XT::to_f32((uint16_t)(v[j] >> 16)), XT::to_f32((uint16_t)(w[j] >> 16)), a);
      }
    }
    a = team_sum(a, 64);
    if (lane == 0) logit[e] = a;
  }
  __syncthreads();
  if (wave != 0) return;
  uint64_t key[kMaxExperts / 64];
#pragma unroll
  for (int j = 0; j < kMaxExperts / 64; ++j) {
    const int e = 64 * j + lane;
    key[j] = e < E ? ((uint64_t)order_key(logit[e]) << 32) | (uint32_t)(0xFFFFFFFFu - (uint32_t)e) : 0u;
  }
  uint32_t chosen = 0;  // bit j: expert 64 j + lane
  for (int i = 0; i < top_k; ++i) {
    uint64_t best = 0;
#pragma unroll
    for (int j = 0; j < kMaxExperts / 64; ++j)
      if (!(chosen >> j & 1) && key[j] > best) best = key[j];
    best = wave_max64(best);
#pragma unroll
    for (int j = 0; j < kMaxExperts / 64; ++j)
      if (key[j] == best) chosen |= 1u << j;
  }
  float m = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < kMaxExperts / 64; ++j)
    if (chosen >> j & 1) m = fmaxf(m, logit[64 * j + lane]);
  m = team_max(m, 64);
  float p[kMaxExperts / 64], sum = 0.0f;
#pragma unroll
  for (int j = 0; j < kMaxExperts / 64; ++j) {
    p[j] = (chosen >> j & 1) ? expf(logit[64 * j + lane] - m) : 0.0f;
    sum += p[j];
  }
  sum = team_sum(sum, 64);
#pragma unroll
  for (int j = 0; j < kMaxExperts / 64; ++j) {
    const int e = 64 * j + lane;
    if (e < E) shares[e * kMaxTokens + t] = (chosen >> j & 1) ? p[j] / sum : kNotChosen;
  }
}

// Tokens of expert e, as a mask of T bits.
__device__ inline uint64_t expert_tokens(const float* __restrict__ shares, int e, int tokens, int lane) {
  const float p = lane < tokens ? shares[e * kMaxTokens + lane] : kNotChosen;
  return __ballot(p != kNotChosen);
}

// Workgroup (i, e): columns [32 i, 32 i + 32) of h for expert e.
template <int TC>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(const uint8_t* __restrict__ xp,
                                                          const uint32_t* __restrict__ xs,
                                                          const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales,
                                                          const float* __restrict__ shares, int H, int I,
                                                          uint8_t* __restrict__ hp, uint32_t* __restrict__ hs) {
  constexpr int NT = 4;  // 2 tiles of gate rows, 2 of up rows
  __shared__ float part[kWaves][NT][64][4];
  __shared__ float hbuf[kChunk][kMxBlock + 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = blockIdx.y, i0 = (int)blockIdx.x * kMxBlock;
  const uint64_t mask = expert_tokens(shares, e, TC * kChunk, lane);
  if (mask == 0) return;
  const int nblk = H / kMxBlock, ksteps = (H + 127) / 128, hsteps = (I + 127) / 128;
  const int r = lane & 15, q = lane >> 4;
  int64_t row[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    row[j] = ((int64_t)e * 2 * I + (j >= 2 ? I : 0) + i0 + (j & 1) * 16 + r) * nblk;
  auto load = [&](MxWeights<NT>& w, int ks) {
    int b = 4 * ks + q;
    b = b < nblk ? b : nblk - 1;  // past the row: the activations are zeros there
    int64_t at[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) at[j] = row[j] + b;
    mx_load_weights(w, codes, scales, at);
  };
  float4_t acc[TC][NT] = {};
  auto multiply = [&](const MxWeights<NT>& w, int ks) {
#pragma unroll
    for (int c = 0; c < TC; ++c) {
      if (!(mask >> (kChunk * c) & 0xFFFFu)) continue;
      MxActivations a;
      const int64_t f = (int64_t)c * ksteps + ks;
      mx_load_activations(a, xp + f * kMxFragBytes, xs + f * 64, lane);
      mx_multiply<NT>(acc[c], a, w);
    }
  };
  MxWeights<NT> w[2];
  int ks = wave;
  if (ks < ksteps) load(w[0], ks);
  for (; ks < ksteps; ks += 2 * kWaves) {
    if (ks + kWaves < ksteps) load(w[1], ks + kWaves);
    multiply(w[0], ks);
    if (ks + 2 * kWaves < ksteps) load(w[0], ks + 2 * kWaves);
    if (ks + kWaves < ksteps) multiply(w[1], ks + kWaves);
  }

#pragma unroll
  for (int c = 0; c < TC; ++c) {
    if (!(mask >> (kChunk * c) & 0xFFFFu)) continue;
#pragma unroll
    for (int j = 0; j < NT; ++j) *reinterpret_cast<float4_t*>(part[wave][j][lane]) = acc[c][j];
    __syncthreads();
    // thread: token tm of the chunk, column tn of 32 (512 threads)
    const int tm = threadIdx.x >> 5, tn = threadIdx.x & 31;
    const int sl = (tm >> 2) * 16 + (tn & 15);
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w8 = 0; w8 < kWaves; ++w8) {
      g += part[w8][tn >> 4][sl][tm & 3];
      u += part[w8][2 + (tn >> 4)][sl][tm & 3];
    }
    const int t = c * kChunk + tm;
    const bool mine = mask >> t & 1;
    const float p = mine ? shares[e * kMaxTokens + t] : 0.0f;
    hbuf[tm][tn] = mine ? p * (g / (1.0f + expf(-g))) * u : 0.0f;
    __syncthreads();
    // 16 threads split a token's block each; behind the last block of h the
    // rest of its K step is zeros
    const int blk = i0 / kMxBlock, last = blk == I / kMxBlock - 1 ? 4 * hsteps - blk : 1;
    if ((int)threadIdx.x < kChunk * last) {
      const int m = threadIdx.x & 15, bb = blk + (int)(threadIdx.x >> 4);
      float v[kMxBlock];
#pragma unroll
      for (int k = 0; k < kMxBlock; ++k) v[k] = bb == blk ? hbuf[m][k] : 0.0f;
      const int64_t f = ((int64_t)e * TC + c) * hsteps + bb / 4;
      mx_store_pieces(mx_split(v), hp + f * kMxFragBytes, hs + f * 64, (bb % 4) * kChunk + m);
    }
    __syncthreads();
  }
}

// Workgroup: columns [16 b, 16 b + 16) of y for all tokens.
template <class YT, int TC>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(const uint8_t* __restrict__ hp,
                                                            const uint32_t* __restrict__ hs,
                                                            const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales,
                                                            const float* __restrict__ shares, int T, int H, int I,
                                                            int E, uint16_t* __restrict__ Y) {
  __shared__ uint64_t tokens[kMaxExperts];
  __shared__ int list[kMaxExperts];
  __shared__ int count;
  __shared__ float part[kWaves][64][4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int e = wave; e < E; e += kWaves) {
    const uint64_t m = expert_tokens(shares, e, TC * kChunk, lane);
    if (lane == 0) tokens[e] = m;
  }
  __syncthreads();
  if (wave == 0) {  // the chosen experts in ascending order
    int n = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const bool on = e0 + lane < E && tokens[e0 + lane] != 0;
      const uint64_t b = __ballot(on);
      if (on) list[n + __popcll(b & ((1ull << lane) - 1))] = e0 + lane;
      n += __popcll(b);
    }
    if (lane == 0) count = n;
  }
  __syncthreads();
  const int nblk = I / kMxBlock, hsteps = (I + 127) / 128;
  const int total = count * hsteps;
  const int r = lane & 15, q = lane >> 4, n0 = (int)blockIdx.x * 16;
  auto load = [&](MxWeights<1>& w, int i) {
    const int e = list[i / hsteps], ks = i % hsteps;
    int b = 4 * ks + q;
    b = b < nblk ? b : nblk - 1;
    const int64_t at[1] = {((int64_t)e * H + n0 + r) * nblk + b};
    mx_load_weights(w, codes, scales, at);
  };
  float4_t acc[TC][1] = {};
  auto multiply = [&](const MxWeights<1>& w, int i) {
    const int e = list[i / hsteps], ks = i % hsteps;
    const uint64_t mask = tokens[e];
#pragma unroll
    for (int c = 0; c < TC; ++c) {
      if (!(mask >> (kChunk * c) & 0xFFFFu)) continue;
      MxActivations a;
      const int64_t f = ((int64_t)e * TC + c) * hsteps + ks;
      mx_load_activations(a, hp + f * kMxFragBytes, hs + f * 64, lane);
      mx_multiply<1>(acc[c], a, w);
    }
  };
  MxWeights<1> w[2];
  int i = wave;
  if (i < total) load(w[0], i);
  for (; i < total; i += 2 * kWaves) {
    if (i + kWaves < total) load(w[1], i + kWaves);
    multiply(w[0], i);
    if (i + 2 * kWaves < total) load(w[0], i + 2 * kWaves);
    if (i + kWaves < total) multiply(w[1], i + kWaves);
  }
#pragma unroll
  for (int c = 0; c < TC; ++c) {
    *reinterpret_cast<float4_t*>(part[wave][lane]) = acc[c][0];
    __syncthreads();
    if (threadIdx.x < 256) {
      const int tm = threadIdx.x >> 4, tn = threadIdx.x & 15;
      const int sl = (tm >> 2) * 16 + tn;
      float v = 0.0f;
#pragma unroll
      for (int w8 = 0; w8 < kWaves; ++w8) v += part[w8][sl][tm & 3];
      const int t = c * kChunk + tm;
      if (t < T) Y[(int64_t)t * H + n0 + tn] = YT::from_f32(v);
    }
    __syncthreads();
  }
}

struct Layout {
  int64_t chunks, xfrags, hfrags;
  size_t shares, xp, xs, hp, hs, bytes;
};
Layout layout(int64_t T, int64_t H, int64_t I, int64_t E) {
  Layout l;
  l.chunks = T <= 16 ? 1 : (T <= 32 ? 2 : 4);
  l.xfrags = l.chunks * ((H + 127) / 128);
  l.hfrags = E * l.chunks * ((I + 127) / 128);
  l.shares = 0;
  l.xp = l.shares + (size_t)E * kMaxTokens * 4;
  l.xs = l.xp + (size_t)l.xfrags * kMxFragBytes;
  l.hp = l.xs + (size_t)l.xfrags * kMxFragScaleBytes;
  l.hs = l.hp + (size_t)l.hfrags * kMxFragBytes;
  l.bytes = l.hs + (size_t)l.hfrags * kMxFragScaleBytes;
  return l;
}

template <class XT, int TC>
hipError_t launch(const uint16_t* X, const uint16_t* router, const uint8_t* up_codes, const uint8_t* up_scales,
                  const uint8_t* down_codes, const uint8_t* down_scales, int T, int H, int I, int E, int top_k,
                  uint16_t* Y, uint8_t* ws, const Layout& l, hipStream_t stream) {
  float* const shares = reinterpret_cast<float*>(ws + l.shares);
  uint32_t* const xs = reinterpret_cast<uint32_t*>(ws + l.xs);
  uint32_t* const hs = reinterpret_cast<uint32_t*>(ws + l.hs);
  moe_route_kernel<XT><<<TC * kChunk, kRouteThreads, 0, stream>>>(X, router, T, H, E, top_k, shares, ws + l.xp, xs);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  moe_up_kernel<TC><<<dim3((unsigned)(I / kMxBlock), (unsigned)E), kThreads, 0, stream>>>(
      ws + l.xp, xs, up_codes, up_scales, shares, H, I, ws + l.hp, hs);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  moe_down_kernel<XT, TC><<<(unsigned)(H / 16), kThreads, 0, stream>>>(ws + l.hp, hs, down_codes, down_scales, shares,
                                                                       T, H, I, E, Y);
  return hipGetLastError();
}

}  // namespace

int mxfp4_moe_max_tokens() { return kMaxTokens; }
int mxfp4_moe_max_experts() { return kMaxExperts; }

size_t mxfp4_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E) { return layout(T, H, I, E).bytes; }

hipError_t launch_mxfp4_moe(const void* X, int xdtype, const void* router, const void* up_codes,
                            const void* up_scales, const void* down_codes, const void* down_scales, int64_t T,
                            int64_t H, int64_t I, int64_t E, int top_k, void* Y, void* workspace, hipStream_t stream) {
  const Layout l = layout(T, H, I, E);
  auto run = [&](auto tag, auto tc) {
    return launch<decltype(tag), decltype(tc)::value>(
        static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(router), static_cast<const uint8_t*>(up_codes),
        static_cast<const uint8_t*>(up_scales), static_cast<const uint8_t*>(down_codes),
        static_cast<const uint8_t*>(down_scales), (int)T, (int)H, (int)I, (int)E, top_k, static_cast<uint16_t*>(Y),
        static_cast<uint8_t*>(workspace), l, stream);
  };
  auto chunks = [&](auto tag) {
    return l.chunks == 1   ? run(tag, std::integral_constant<int, 1>{})
           : l.chunks == 2 ? run(tag, std::integral_constant<int, 2>{})
                           : run(tag, std::integral_constant<int, 4>{});
  };
  return xdtype == 0 ? chunks(F16{}) : chunks(BF16{});
}

}  // namespace woq
