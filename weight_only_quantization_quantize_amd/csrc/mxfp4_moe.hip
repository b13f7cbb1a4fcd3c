// A mixture-of-experts layer on T <= 64 tokens with microscaled 4-bit experts:
//   logits[t, e] = sum_k x[t, k] router[e, k]                      (fp32)
//   S(t) = the top_k experts by (logit descending, index ascending)
//   p[t, e] = exp(logits[t, e]) / sum over S(t) of exp(logits[t, .])   for e in S(t)
//   h[t, e, i] = silu(x[t] . up[e, i]) (x[t] . up[e, I + i])        silu(g) = g / (1 + exp(-g))
//   y[t] = sum over S(t) of p[t, e] (down[e] h[t, e])               rounded once
//
// At a few tokens the layer is bound by streaming the chosen experts' weights
// (3 I H 17/32 bytes each) once, so an expert's weights are read once for up to
// 16 of its tokens, 16 weight rows at a time against those tokens on the matrix
// units (mxfp4_stream.h); each further 16 tokens take a turn of their own, out of
// L2.  (All chunks in one turn needs 64 sums a lane more and spilled.)
//
// Four launches:
//   route   logits, one workgroup per expert and 8 tokens; x split into pieces
//   choose  one workgroup: the tokens' experts and shares, and the list of turns
//           (an expert and up to 16 of its tokens, in ascending order)
//   up      one workgroup per (turn, 32 columns of h): gate and up rows, then
//           p silu(g) u, split into pieces again (14 bits of a block's largest
//           magnitude).  The share is folded in here, where the values are still
//           fp32, so that the next product adds over experts by itself.
//   down    one workgroup per 16 columns of y, over all turns: each wave adds its
//           products into a sum per token in LDS of its own, and the waves' sums
//           are added in a fixed order (no atomics).
// Working the choice out in every workgroup of the up launch instead of in a
// launch of its own took 4 us there for one token and 15 for five.
#include "mxfp4_stream.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kChunk = 16;
constexpr int kMaxTokens = 64;
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 64;
constexpr int kMaxTurns = kMaxExperts + kMaxTokens * kMaxTopK / 16;
constexpr int kRouteThreads = 512;
constexpr int kRouteTokens = 8;   // tokens per workgroup of the logits
constexpr int kChooseWaves = 16;
constexpr int kUpWaves = 8;         // at most
constexpr int kDownWaves = 8;

// An expert and up to 16 of its tokens.
struct Turn {
  int expert, count;
  float share[kChunk];
  uint8_t token[kChunk];
};
struct Plan {
  int turns;
  int pad[3];
};

// A logit's order as an unsigned number; the zeros are equal and a NaN comes
// below -infinity.
__device__ inline uint32_t order_key(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ inline float key_value(uint32_t k) {
  return __builtin_bit_cast(float, k == 0 ? 0x7FC00000u : ((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k));
}

__device__ inline uint32_t wave_max(uint32_t v) {
  auto step = [&](auto ctrl, auto rows) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
    v = v > o ? v : o;
  };
  step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xF>{});  // row_shr 1, 2, 4, 8
  step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});  // row_bcast 15, 31
  step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// logits [64][E].  Workgroups [0, groups E) compute logits, the rest split x
// (fragments of 16 rows, super-step order).
template <class XT, int TOKENS>
__global__ __launch_bounds__(kRouteThreads) void moe_route_kernel(const uint16_t* __restrict__ X,
                                                                  const uint16_t* __restrict__ router, int T, int H,
                                                                  int E, int groups, float* __restrict__ logits,
                                                                  uint8_t* __restrict__ xp, uint32_t* __restrict__ xs) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if ((int)blockIdx.x >= groups * E) {
    const int supers = (H + 511) / 512;
    const int i = ((int)blockIdx.x - groups * E) * kRouteThreads + (int)threadIdx.x;  // block of x
    const int t = i / (kSuper * supers), b = i % (kSuper * supers);
    if (t >= T) return;
    float v[kMxBlock] = {};
    if (b * kMxBlock < H) mx_load_block<XT>(X + (int64_t)t * H + b * kMxBlock, v);
    const int64_t f = ((int64_t)(t / kChunk) * supers + b / kSuper) * 4 + b % 4;
    mx_store_pieces(mx_split(v), xp + f * kMxFragBytes, xs + f * 64, (b % kSuper / 4) * kChunk + t % kChunk);
    return;
  }
  __shared__ float part[kRouteThreads / 64][TOKENS];
  const int e = (int)blockIdx.x / groups, t0 = (int)blockIdx.x % groups * TOKENS;
  const int n = T - t0 < TOKENS ? T - t0 : TOKENS;
  float a[TOKENS] = {};
  for (int k = (int)threadIdx.x * 8; k < H; k += kRouteThreads * 8) {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(router + (int64_t)e * H + k);
    u32x4_t v[TOKENS];
#pragma unroll
    for (int t = 0; t < TOKENS; ++t)
      v[t] = *reinterpret_cast<const u32x4_t*>(X + (int64_t)(t0 + (t < n ? t : n - 1)) * H + k);
#pragma unroll
    for (int t = 0; t < TOKENS; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[t] = fmaf(XT::to_f32((uint16_t)(v[t][j] & 0xFFFFu)), XT::to_f32((uint16_t)(w[j] & 0xFFFFu)), a[t]);
        a[t] = fmaf(XT::to_f32((uint16_t)(v[t][j] >> 16)), XT::to_f32((uint16_t)(w[j] >> 16)), a[t]);
      }
  }
#pragma unroll
  for (int t = 0; t < TOKENS; ++t) {
    const float s = team_sum(a[t], 64);
    if (lane == 0) part[wave][t] = s;
  }
  __syncthreads();
  if ((int)threadIdx.x < n) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kRouteThreads / 64; ++w) s += part[w][threadIdx.x];
    logits[(t0 + (int)threadIdx.x) * E + e] = s;
  }
}

// One workgroup.  logits [T][E] -> the plan and its turns.
// NJ: lanes' experts, 64 NJ >= E.
template <int NJ>
__global__ __launch_bounds__(kChooseWaves * 64) void moe_choose_kernel(const float* __restrict__ logits, int T, int E,
                                                                       int top_k, Plan* __restrict__ plan,
                                                                       Turn* __restrict__ turns) {
  __shared__ uint16_t ids[kMaxTokens * kMaxTopK];      // [token][choice]
  __shared__ float shares[kMaxTokens * kMaxTopK];
  __shared__ unsigned long long tokens[kMaxExperts];   // of an expert
  __shared__ uint16_t base[kMaxExperts];               // its first turn
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int e = threadIdx.x; e < E; e += kChooseWaves * 64) tokens[e] = 0;
  __syncthreads();
  constexpr int kTokens = kMaxTokens / kChooseWaves;  // of a wave, at most
  float logit[kTokens][NJ];                           // of expert 64 j + lane
#pragma unroll
  for (int i = 0; i < kTokens; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int t = wave + kChooseWaves * i, e = 64 * j + lane;
      logit[i][j] = t < T && e < E ? logits[t * E + e] : 0.0f;
    }
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int t = wave + kChooseWaves * i;
    if (t >= T) break;
    uint32_t key[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) key[j] = 64 * j + lane < E ? order_key(logit[i][j]) : 0u;
    uint32_t taken = 0;  // bit j: expert 64 j + lane
    for (int c = 0; c < top_k; ++c) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (!(taken >> j & 1) && key[j] > m) m = key[j];
      m = wave_max(m);
      int id = -1;  // the lowest index of that key
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (id < 0) {
          const uint64_t b = __ballot(!(taken >> j & 1) && key[j] == m && 64 * j + lane < E);
          if (b) id = 64 * j + __builtin_ctzll(b);
        }
      if (lane == (id & 63)) taken |= 1u << (id >> 6);
      if (lane == 0) {
        ids[t * top_k + c] = (uint16_t)id;
        shares[t * top_k + c] = key_value(m);
        atomicOr(&tokens[id], 1ull << t);
      }
    }
    // softmax over the choices, one a lane
    const float w = lane < top_k ? expf(shares[t * top_k + lane] - shares[t * top_k]) : 0.0f;
    const float sum = team_sum(w, 64);
    if (lane < top_k) shares[t * top_k + lane] = w / sum;
  }
  __syncthreads();
  if (wave == 0) {  // turns before each expert's
    int at = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const int n = e < E ? (__popcll(tokens[e]) + kChunk - 1) / kChunk : 0;
      int upto = n;
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(upto, off, 64);
        if (lane >= off) upto += o;
      }
      if (e < E) base[e] = (uint16_t)(at + upto - n);
      at += __shfl(upto, 63, 64);
    }
    if (lane == 0) plan->turns = at;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kChooseWaves * 64) {
    const int n = __popcll(tokens[e]);
    for (int c = 0; c * kChunk < n; ++c) {
      Turn& r = turns[base[e] + c];
      r.expert = e;
      r.count = n - c * kChunk < kChunk ? n - c * kChunk : kChunk;
    }
  }
  for (int i = threadIdx.x; i < T * top_k; i += kChooseWaves * 64) {
    const int t = i / top_k, e = ids[i];
    const int row = __popcll(tokens[e] & ((1ull << t) - 1));
    Turn& r = turns[base[e] + row / kChunk];
    r.share[row % kChunk] = shares[i];
    r.token[row % kChunk] = (uint8_t)t;
  }
}

// Workgroup (i, turn): columns [32 i, 32 i + 32) of h for the turn's tokens.
__global__ __launch_bounds__(kUpWaves * 64, 3) void moe_up_kernel(const uint8_t* __restrict__ xp,
                                                                  const uint8_t* __restrict__ xs,
                                                                  const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales,
                                                                  const Plan* __restrict__ plan,
                                                                  const Turn* __restrict__ turns, int H, int I, int E,
                                                                  uint8_t* __restrict__ hp, uint32_t* __restrict__ hs) {
  constexpr int NT = 4;  // gate rows, up rows, gate rows, up rows
  __shared__ __attribute__((aligned(16))) uint8_t stage_all[kUpWaves][kUnitStage];
  __shared__ float hbuf[kChunk][kMxBlock + 1];
  static_assert(NT * 1024 <= kUnitStage, "a wave's partial sums fit its stage's place");

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int turn = blockIdx.y, i0 = (int)blockIdx.x * kMxBlock;
  if (turn >= plan->turns) return;
  const Turn& rec = turns[turn];
  const int e = rec.expert, count = rec.count;

  const int nblk = H / kMxBlock, supers = (H + 511) / 512, hsupers = (I + 511) / 512;
  const int64_t rows_left = (int64_t)E * 2 * I - ((int64_t)e * 2 * I + i0);
  const uint8_t* const wcodes = codes + ((int64_t)e * 2 * I + i0) * nblk * 16;
  const uint8_t* const wscales = scales + ((int64_t)e * 2 * I + i0) * nblk;
  const int waves = blockDim.x >> 6;  // wave w takes super-steps w, w + waves, ...
  uint8_t* const stage = stage_all[wave];
  // tiles in the order gate, up, gate, up; two units in flight, loaded in order;
  // past the end a line or two of the first rows is loaded in their place
  MxUnit u[2];
  auto row_of = [&](int j) { return (j & 1 ? I : 0) + (j >> 1) * 16; };
  auto ahead = [&](int j, int S_) {
    const bool more = S_ < supers;
    const int S = more ? S_ : 0;
    const int64_t row = more ? row_of(j) : 0;
    __builtin_amdgcn_sched_barrier(0);
    mx_load_unit(u[j & 1], wcodes + row * nblk * 16, wscales + row * nblk, 15, (rows_left - row) * nblk, more ? nblk : 1, S, lane);
    __builtin_amdgcn_sched_barrier(0);
  };
  float4_t acc[NT] = {};
  int S = wave;
  // rows past the turn's last token repeat it
  const int t = rec.token[(lane & 15) < count ? lane & 15 : count - 1];
  const MxPlace place = mx_place(t / kChunk * supers * 4, (lane & 48) + t % kChunk);
  ahead(0, S);
  ahead(1, S);
  for (; S < supers; S += waves) {
    MxActivations a[4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
      mx_load_activations(a[s], xp + (int64_t)(S * 4 + s) * kMxFragBytes, xs + (int64_t)(S * 4 + s) * kMxFragScaleBytes, place);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      mx_stage_unit(u[j & 1], stage, 15, (rows_left - row_of(j)) * nblk, nblk, S, lane);
      ahead((j + 2) & 3, j < 2 ? S : S + waves);
      const int sc = mx_staged_scale(stage, lane);
      mx_each_step([&](auto sel) {
        constexpr int s = decltype(sel)::value;
        mx_multiply<s>(acc[j], a[s], mx_staged_weights(stage, s, lane), sc);
      });
    }
  }
  // the waves' partial sums meet in the stages' place, [tile][lane][4] a wave
#pragma unroll
  for (int j = 0; j < NT; ++j) *reinterpret_cast<float4_t*>(stage + (j * 64 + lane) * 16) = acc[j];
  __syncthreads();
  for (int o = threadIdx.x; o < kChunk * kMxBlock; o += (int)blockDim.x) {
    const int tm = o >> 5, tn = o & 31;
    const int sl = (tm >> 2) * 16 + (tn & 15);
    float g = 0.0f, v = 0.0f;
    for (int w = 0; w < waves; ++w) {
      const float* const part = reinterpret_cast<const float*>(stage_all[w]);
      g += part[((tn >> 4) * 128 + sl) * 4 + (tm & 3)];
      v += part[((tn >> 4) * 128 + 64 + sl) * 4 + (tm & 3)];
    }
    hbuf[tm][tn] = tm < count ? rec.share[tm] * (g / (1.0f + expf(-g))) * v : 0.0f;
  }
  __syncthreads();
  // 16 threads split a row's block each; behind the last block of h the rest of
  // its super-step is zeros
  const int blk = i0 / kMxBlock, last = blk == I / kMxBlock - 1 ? kSuper * hsupers - blk : 1;
  for (int o = threadIdx.x; o < kChunk * last; o += (int)blockDim.x) {
    const int m = o & 15, b = blk + (o >> 4);
    float v[kMxBlock];
#pragma unroll
    for (int k = 0; k < kMxBlock; ++k) v[k] = b == blk ? hbuf[m][k] : 0.0f;
    const int64_t f = ((int64_t)turn * hsupers + b / kSuper) * 4 + b % 4;
    mx_store_pieces(mx_split(v), hp + f * kMxFragBytes, hs + f * 64, (b % kSuper / 4) * kChunk + m);
  }
}

// Workgroup: columns [16 b, 16 b + 16) of y for all tokens.
template <class YT, int TC>
__global__ __launch_bounds__(kDownWaves * 64) void moe_down_kernel(const uint8_t* __restrict__ hp,
                                                                   const uint8_t* __restrict__ hs,
                                                                   const uint8_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scales,
                                                                   const Plan* __restrict__ plan,
                                                                   const Turn* __restrict__ turns, int T, int H, int I,
                                                                   int E, uint16_t* __restrict__ Y) {
  constexpr int kRows = TC * kChunk;
  __shared__ __attribute__((aligned(16))) uint8_t stage_all[kDownWaves][kUnitStage];
  __shared__ float sums[kDownWaves][kRows][kChunk + 1];
  __shared__ uint32_t table[kMaxTurns];  // expert + count << 16
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nblk = I / kMxBlock, supers = (I + 511) / 512;
  const int nturns = plan->turns, units = nturns * supers;
  const int n0 = (int)blockIdx.x * 16;
  uint8_t* const stage = stage_all[wave];
  for (int k = threadIdx.x; k < nturns; k += kDownWaves * 64) table[k] = (uint32_t)turns[k].expert | (uint32_t)turns[k].count << 16;
  for (int o = lane; o < kRows * (kChunk + 1); o += 64) (&sums[wave][0][0])[o] = 0.0f;
  __syncthreads();
  // the wave's run of units: a turn's super-steps follow one another
  const int u0 = (int)((int64_t)units * wave / kDownWaves), u1 = (int)((int64_t)units * (wave + 1) / kDownWaves);
  struct Work {
    MxUnit u;
    MxActivations a[4];
    uint32_t token;  // of rows 4 q .. 4 q + 3
  };
  auto load = [&](Work& w, int i) {
    const int k = i / supers, S = i % supers;
    const uint32_t rec = (uint32_t)__builtin_amdgcn_readfirstlane((int)table[k]);
    const int64_t row = (int64_t)(rec & 0xFFFFu) * H + n0;
    mx_load_unit(w.u, codes + row * nblk * 16, scales + row * nblk, 15, ((int64_t)E * H - row) * nblk, nblk, S, lane);
    // rows past the turn's tokens are left as they are: their sums are not taken
    if ((lane & 15) < (int)(rec >> 16)) {
      const MxPlace place = mx_place(0, lane);
      const int64_t f = ((int64_t)k * supers + S) * 4;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        mx_load_activations(w.a[s], hp + (f + s) * kMxFragBytes, hs + (f + s) * kMxFragScaleBytes, place);
    }
    w.token = reinterpret_cast<const uint32_t*>(turns[k].token)[lane >> 4];
  };
  float4_t acc = {};
  auto work = [&](const Work& w, int i) {
    const int k = i / supers, S = i % supers;
    const uint32_t rec = (uint32_t)__builtin_amdgcn_readfirstlane((int)table[k]);
    const int64_t row = (int64_t)(rec & 0xFFFFu) * H + n0;
    mx_stage_unit(w.u, stage, 15, ((int64_t)E * H - row) * nblk, nblk, S, lane);
    const int sc = mx_staged_scale(stage, lane);
    mx_each_step([&](auto sel) {
      constexpr int s = decltype(sel)::value;
      mx_multiply<s>(acc, w.a[s], mx_staged_weights(stage, s, lane), sc);
    });
    if (S == supers - 1 || i + 1 == u1) {  // the wave is through with the turn
      const int count = (int)(rec >> 16);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * (lane >> 4) + e < count) sums[wave][w.token >> (8 * e) & 63u][lane & 15] += acc[e];
      acc = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
  };
  Work a = {}, b = {};
  if (u0 < u1) load(a, u0);
  if (u0 + 1 < u1) load(b, u0 + 1);
  for (int i = u0; i < u1; i += 2) {
    work(a, i);
    if (i + 2 < u1) load(a, i + 2);
    if (i + 1 < u1) work(b, i + 1);
    if (i + 3 < u1) load(b, i + 3);
  }
  __syncthreads();
  for (int o = threadIdx.x; o < T * kChunk; o += kDownWaves * 64) {
    const int t = o / kChunk, n = o % kChunk;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kDownWaves; ++w) v += sums[w][t][n];
    Y[(int64_t)t * H + n0 + n] = YT::from_f32(v);
  }
}

struct Layout {
  int64_t turns, xfrags, hfrags;
  size_t logits, plan, records, xp, xs, hp, hs, bytes;
};
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
Layout layout(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k) {
  Layout l;
  // a turn for each chosen expert and one for each further 16 tokens of it
  l.turns = (T * top_k < E ? T * top_k : E) + T * top_k / kChunk;
  l.xfrags = (T + kChunk - 1) / kChunk * ((H + 511) / 512 * 4);
  l.hfrags = l.turns * ((I + 511) / 512 * 4);
  l.logits = 0;
  l.plan = up256((size_t)E * T * 4);
  l.records = l.plan + 256;
  l.xp = up256(l.records + (size_t)l.turns * sizeof(Turn));
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
  float* const logits = reinterpret_cast<float*>(ws + l.logits);
  Plan* const plan = reinterpret_cast<Plan*>(ws + l.plan);
  Turn* const turns = reinterpret_cast<Turn*>(ws + l.records);
  uint8_t* const xs = ws + l.xs;
  uint8_t* const hs = ws + l.hs;
  const int tokens = T == 1 ? 1 : kRouteTokens;
  const int groups = (T + tokens - 1) / tokens;
  const int blocks = T * kSuper * ((H + 511) / 512);
  const unsigned grid = (unsigned)(groups * E + (blocks + kRouteThreads - 1) / kRouteThreads);
  if (T == 1)
    moe_route_kernel<XT, 1><<<grid, kRouteThreads, 0, stream>>>(X, router, T, H, E, groups, logits, ws + l.xp,
                                                                reinterpret_cast<uint32_t*>(xs));
  else
    moe_route_kernel<XT, kRouteTokens><<<grid, kRouteThreads, 0, stream>>>(X, router, T, H, E, groups, logits, ws + l.xp,
                                                                           reinterpret_cast<uint32_t*>(xs));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (E <= 64)
    moe_choose_kernel<1><<<1, kChooseWaves * 64, 0, stream>>>(logits, T, E, top_k, plan, turns);
  else
    moe_choose_kernel<kMaxExperts / 64><<<1, kChooseWaves * 64, 0, stream>>>(logits, T, E, top_k, plan, turns);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  // a wave for every super-step of a row, up to 8: all loads of a row tile start at once
  const int supers = (H + 511) / 512, waves = supers < kUpWaves ? supers : kUpWaves;
  moe_up_kernel<<<dim3((unsigned)(I / kMxBlock), (unsigned)l.turns), (unsigned)(waves * 64), 0, stream>>>(
      ws + l.xp, xs, up_codes, up_scales, plan, turns, H, I, E, ws + l.hp, reinterpret_cast<uint32_t*>(hs));
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  moe_down_kernel<XT, TC><<<(unsigned)(H / 16), kDownWaves * 64, 0, stream>>>(ws + l.hp, hs, down_codes, down_scales,
                                                                             plan, turns, T, H, I, E, Y);
  return hipGetLastError();
}

}  // namespace

int mxfp4_moe_max_tokens() { return kMaxTokens; }
int mxfp4_moe_max_experts() { return kMaxExperts; }
int mxfp4_moe_max_top_k() { return kMaxTopK; }

size_t mxfp4_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k) {
  return layout(T, H, I, E, top_k).bytes;
}

hipError_t launch_mxfp4_moe(const void* X, int xdtype, const void* router, const void* up_codes,
                            const void* up_scales, const void* down_codes, const void* down_scales, int64_t T,
                            int64_t H, int64_t I, int64_t E, int top_k, void* Y, void* workspace, hipStream_t stream) {
  const Layout l = layout(T, H, I, E, top_k);
  auto run = [&](auto tag, auto tc) {
    return launch<decltype(tag), decltype(tc)::value>(
        static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(router), static_cast<const uint8_t*>(up_codes),
        static_cast<const uint8_t*>(up_scales), static_cast<const uint8_t*>(down_codes),
        static_cast<const uint8_t*>(down_scales), (int)T, (int)H, (int)I, (int)E, top_k, static_cast<uint16_t*>(Y),
        static_cast<uint8_t*>(workspace), l, stream);
  };
  auto chunks = [&](auto tag) {
    return T <= 16   ? run(tag, std::integral_constant<int, 1>{})
           : T <= 32 ? run(tag, std::integral_constant<int, 2>{})
                     : run(tag, std::integral_constant<int, 4>{});
  };
  return xdtype == 0 ? chunks(F16{}) : chunks(BF16{});
}

}  // namespace woq
