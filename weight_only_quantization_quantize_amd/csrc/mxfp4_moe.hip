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
// Three launches:
//   route  logits, one workgroup per expert and 8 tokens; x split into pieces
//   up     one workgroup per (chosen expert, 32 columns of h).  Each works out
//          the choice from the logits itself, which takes less than a launch
//          would: where the tokens choose fewer experts than there are
//          (T top_k < E), waves choose for a token each and the workgroup takes
//          the slot-th chosen expert; otherwise a slot is an expert and only its
//          rank among the logits is counted, a token a lane.  Gate and up rows,
//          then w silu(g) u with w = exp(logit - max), split into pieces again
//          (14 bits of a block's largest magnitude), one row per token of the
//          expert.  The weight is folded in here, where the values are still
//          fp32, so that the next product adds over experts by itself.
//   down   one workgroup per 16 columns of y, over all slots: each wave adds its
//          products into a sum per token in LDS of its own, the waves' sums are
//          added in a fixed order (no atomics) and divided by the sum of w.
#include "mxfp4_stream.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kChunk = 16;
constexpr int kMaxTokens = 64;
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 64;
constexpr int kMaxTurns = 4 * kMaxExperts;
constexpr int kRouteThreads = 256;
constexpr int kRouteTokens = 8;   // tokens per workgroup of the logits
constexpr int kUpWaves = 4;
constexpr int kDownWaves = 8;

// What the up launch leaves for the down launch about a slot.
struct Slot {
  int expert, count;          // its tokens
  float w[kMaxTokens];        // their weights, by the order of `token`
  uint8_t token[kMaxTokens];  // ascending
};

// A logit's order as an unsigned number; the zeros are equal and a NaN comes
// below -infinity.
__device__ inline uint32_t order_key(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
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

// logits [E][64].  Workgroups [0, groups E) compute logits, the rest split x
// (fragments of 16 rows, super-step order).
template <class XT>
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
  __shared__ float part[kRouteThreads / 64][kRouteTokens];
  const int e = (int)blockIdx.x / groups, t0 = (int)blockIdx.x % groups * kRouteTokens;
  const int n = T - t0 < kRouteTokens ? T - t0 : kRouteTokens;
  float a[kRouteTokens] = {};
  for (int k = (int)threadIdx.x * 8; k < H; k += kRouteThreads * 8) {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(router + (int64_t)e * H + k);
    u32x4_t v[kRouteTokens];
#pragma unroll
    for (int t = 0; t < kRouteTokens; ++t)
      v[t] = *reinterpret_cast<const u32x4_t*>(X + (int64_t)(t0 + (t < n ? t : n - 1)) * H + k);
#pragma unroll
    for (int t = 0; t < kRouteTokens; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[t] = fmaf(XT::to_f32((uint16_t)(v[t][j] & 0xFFFFu)), XT::to_f32((uint16_t)(w[j] & 0xFFFFu)), a[t]);
        a[t] = fmaf(XT::to_f32((uint16_t)(v[t][j] >> 16)), XT::to_f32((uint16_t)(w[j] >> 16)), a[t]);
      }
  }
#pragma unroll
  for (int t = 0; t < kRouteTokens; ++t) {
    const float s = team_sum(a[t], 64);
    if (lane == 0) part[wave][t] = s;
  }
  __syncthreads();
  if ((int)threadIdx.x < n) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kRouteThreads / 64; ++w) s += part[w][threadIdx.x];
    logits[e * kMaxTokens + t0 + threadIdx.x] = s;
  }
}

// Workgroup (i, slot): columns [32 i, 32 i + 32) of h for the slot's expert.
__global__ __launch_bounds__(kUpWaves * 64, 2) void moe_up_kernel(const uint8_t* __restrict__ xp,
                                                                  const uint32_t* __restrict__ xs,
                                                                  const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales,
                                                                  const float* __restrict__ logits, int T, int H,
                                                                  int I, int E, int top_k, int by_token, int chunks,
                                                                  Slot* __restrict__ slots, uint8_t* __restrict__ hp,
                                                                  uint32_t* __restrict__ hs) {
  constexpr int NT = 4;  // 2 tiles of gate rows, 2 of up rows
  __shared__ __attribute__((aligned(16))) uint8_t stage_all[kUpWaves][NT][kUnitStage];
  __shared__ float hbuf[kChunk][kMxBlock + 1];
  __shared__ uint64_t words[kMaxExperts / 64];            // chosen experts, by token
  __shared__ uint16_t ids[kMaxExperts];                   // [token][choice]: T top_k < E of them
  __shared__ float weight[kMaxTokens];
  __shared__ int ranks[kUpWaves][kMaxTokens];
  __shared__ uint32_t tops[kUpWaves][kMaxTokens];
  __shared__ uint8_t token[kMaxTokens];
  __shared__ uint64_t chosen_by;
  static_assert(kUpWaves * NT * 1024 <= (int)sizeof(stage_all), "the partial sums fit the stages' place");

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slot = blockIdx.y, i0 = (int)blockIdx.x * kMxBlock;

  // The slot's expert, the tokens that chose it and their weights.
  int e = slot;
  if (by_token) {
    if (threadIdx.x < kMaxExperts / 64) words[threadIdx.x] = 0;
    __syncthreads();
    for (int t = wave; t < T; t += kUpWaves) {
      uint32_t key[kMaxExperts / 64];
#pragma unroll
      for (int j = 0; j < kMaxExperts / 64; ++j)
        if (64 * j < E) key[j] = 64 * j + lane < E ? order_key(logits[(64 * j + lane) * kMaxTokens + t]) : 0u;
      uint32_t taken = 0;  // bit j: expert 64 j + lane
      for (int c = 0; c < top_k; ++c) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < kMaxExperts / 64; ++j)
          if (64 * j < E && !(taken >> j & 1) && key[j] > m) m = key[j];
        m = wave_max(m);
        int id = -1;  // the lowest index of that key
#pragma unroll
        for (int j = 0; j < kMaxExperts / 64; ++j) {
          if (64 * j < E && id < 0) {
            const uint64_t b = __ballot(!(taken >> j & 1) && key[j] == m && 64 * j + lane < E);
            if (b) id = 64 * j + __builtin_ctzll(b);
          }
        }
        if (lane == (id & 63)) taken |= 1u << (id >> 6);
        if (lane == 0) {
          ids[t * top_k + c] = (uint16_t)id;
          atomicOr(reinterpret_cast<unsigned long long*>(&words[id >> 6]), 1ull << (id & 63));
        }
      }
    }
    __syncthreads();
    int left = slot;
    e = -1;
    for (int j = 0; j < kMaxExperts / 64 && e < 0; ++j) {
      uint64_t w = words[j];
      const int n = __popcll(w);
      if (left >= n) {
        left -= n;
      } else {
        for (; left > 0; --left) w &= w - 1;
        e = 64 * j + __builtin_ctzll(w);
      }
    }
    e = __builtin_amdgcn_readfirstlane(e);
    if (wave == 0) {
      bool mine = false;
      float w = 0.0f;
      if (lane < T && e >= 0) {
        for (int c = 0; c < top_k; ++c) mine |= ids[lane * top_k + c] == e;
        w = expf(logits[e * kMaxTokens + lane] - logits[(int)ids[lane * top_k] * kMaxTokens + lane]);
      }
      const uint64_t b = __ballot(mine);
      weight[lane] = mine ? w : 0.0f;
      if (lane == 0) chosen_by = b;
    }
  } else {
    // rank of e among the logits of token `lane`, a share of the experts a wave
    const float own = lane < T ? logits[e * kMaxTokens + lane] : 0.0f;
    const uint32_t key = order_key(own);
    int rank = 0;
    uint32_t top = 0;
    float top_logit = 0.0f;
    for (int j = wave; j < E; j += kUpWaves) {
      const uint32_t k = order_key(lane < T ? logits[j * kMaxTokens + lane] : 0.0f);
      rank += (k > key || (k == key && j < e)) ? 1 : 0;
      top = k > top ? k : top;
    }
    ranks[wave][lane] = rank;
    tops[wave][lane] = top;
    __syncthreads();
    if (wave == 0) {
      for (int w = 1; w < kUpWaves; ++w) {
        rank += ranks[w][lane];
        top = tops[w][lane] > top ? tops[w][lane] : top;
      }
      // the logit of that key (all NaN: key 0, and the weight is a NaN)
      top_logit = __builtin_bit_cast(float, top == 0 ? 0x7FC00000u : ((top & 0x80000000u) ? top & 0x7FFFFFFFu : ~top));
      const bool mine = lane < T && rank < top_k;
      const uint64_t b = __ballot(mine);
      weight[lane] = mine ? expf(own - top_logit) : 0.0f;
      if (lane == 0) chosen_by = b;
    }
  }
  __syncthreads();
  const uint64_t mask = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(chosen_by >> 32)) << 32 |
                        (uint32_t)__builtin_amdgcn_readfirstlane((int)chosen_by);
  const int count = __popcll(mask);
  if (wave == 0 && (mask >> lane & 1)) token[__popcll(mask & ((1ull << lane) - 1))] = (uint8_t)lane;
  __syncthreads();
  if (blockIdx.x == 0 && wave == 0) {
    Slot& s = slots[slot];
    if (lane == 0) {
      s.expert = e;
      s.count = count;
    }
    if (lane < count) {
      s.token[lane] = token[lane];
      s.w[lane] = weight[token[lane]];
    }
  }
  if (count == 0) return;

  const int nblk = H / kMxBlock, supers = (H + 511) / 512, hsupers = (I + 511) / 512;
  const int64_t rows_left = (int64_t)E * 2 * I - ((int64_t)e * 2 * I + i0);
  const uint8_t* const wcodes = codes + ((int64_t)e * 2 * I + i0) * nblk * 16;
  const uint8_t* const wscales = scales + ((int64_t)e * 2 * I + i0) * nblk;
  auto tile_row = [&](int j) { return (j >= 2 ? I : 0) + (j & 1) * 16; };
  MxUnit u[NT];
  auto load = [&](int S) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int64_t row = tile_row(j);
      mx_load_unit(u[j], wcodes + row * nblk * 16, wscales + row * nblk, 15, (rows_left - row) * nblk, nblk, S, lane);
    }
  };
  float* const part = reinterpret_cast<float*>(&stage_all[0][0][0]);  // [wave][tile][lane][4]
  // an expert with more than 16 tokens takes another turn over its weights, out of L2
  for (int c = 0; c * kChunk < count; ++c) {
    const int own = c * kChunk + (lane & 15), t = token[own < count ? own : count - 1];
    const MxPlace place = mx_place(t / kChunk * supers * 4, (lane & 48) + t % kChunk);
    float4_t acc[NT] = {};
    int S = wave;
    if (S < supers) load(S);
    for (; S < supers; S += kUpWaves) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
        mx_stage_unit(u[j], stage_all[wave][j], 15, (rows_left - tile_row(j)) * nblk, nblk, S, lane);
      if (S + kUpWaves < supers) load(S + kUpWaves);
      int sc[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) sc[j] = mx_staged_scale(stage_all[wave][j], lane);
      mx_each_step([&](auto sel) {
        constexpr int s = decltype(sel)::value;
        MxActivations a;
        const int64_t f = S * 4 + s;
        mx_load_activations(a, xp + f * kMxFragBytes, reinterpret_cast<const uint8_t*>(xs) + f * kMxFragScaleBytes, place);
#pragma unroll
        for (int j = 0; j < NT; ++j) mx_multiply<s>(acc[j], a, mx_staged_weights(stage_all[wave][j], s, lane), sc[j]);
      });
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j) *reinterpret_cast<float4_t*>(part + ((wave * NT + j) * 64 + lane) * 4) = acc[j];
    __syncthreads();
    // two elements of the 16 x 32 block of h a thread
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const int tm = (int)(threadIdx.x >> 5) + 8 * o, tn = threadIdx.x & 31;
      const int sl = (tm >> 2) * 16 + (tn & 15);
      float g = 0.0f, v = 0.0f;
#pragma unroll
      for (int w = 0; w < kUpWaves; ++w) {
        g += part[((w * NT + (tn >> 4)) * 64 + sl) * 4 + (tm & 3)];
        v += part[((w * NT + 2 + (tn >> 4)) * 64 + sl) * 4 + (tm & 3)];
      }
      const int row = c * kChunk + tm;
      hbuf[tm][tn] = row < count ? weight[token[row]] * (g / (1.0f + expf(-g))) * v : 0.0f;
    }
    __syncthreads();
    // 16 threads split a row's block each; behind the last block of h the rest
    // of its super-step is zeros
    const int blk = i0 / kMxBlock, last = blk == I / kMxBlock - 1 ? kSuper * hsupers - blk : 1;
    if ((int)threadIdx.x < kChunk * last) {
      const int m = threadIdx.x & 15, b = blk + (int)(threadIdx.x >> 4);
      float v[kMxBlock];
#pragma unroll
      for (int k = 0; k < kMxBlock; ++k) v[k] = b == blk ? hbuf[m][k] : 0.0f;
      const int64_t f = (((int64_t)slot * chunks + c) * hsupers + b / kSuper) * 4 + b % 4;
      mx_store_pieces(mx_split(v), hp + f * kMxFragBytes, hs + f * 64, (b % kSuper / 4) * kChunk + m);
    }
  }
}

// Workgroup: columns [16 b, 16 b + 16) of y for all tokens.
template <class YT, int TC>
__global__ __launch_bounds__(kDownWaves * 64) void moe_down_kernel(const uint8_t* __restrict__ hp,
                                                                   const uint32_t* __restrict__ hs,
                                                                   const uint8_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scales,
                                                                   const Slot* __restrict__ slots, int nslots, int T,
                                                                   int H, int I, int E, uint16_t* __restrict__ Y) {
  constexpr int kRows = TC * kChunk, chunks = TC;
  __shared__ __attribute__((aligned(16))) uint8_t stage_all[kDownWaves][kUnitStage];
  __shared__ float sums[kDownWaves][kRows][kChunk + 1];
  __shared__ float total[kRows];
  __shared__ uint16_t list[kMaxExperts], experts[kMaxExperts], counts[kMaxExperts];
  __shared__ uint16_t turn[kMaxTurns];  // (place in the list) * 4 + chunk
  __shared__ int live, turns;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave == 0) {  // the slots that have tokens
    int n = 0;
    for (int s0 = 0; s0 < nslots; s0 += 64) {
      const int c = s0 + lane < nslots ? slots[s0 + lane].count : 0;
      const uint64_t b = __ballot(c > 0);
      if (c > 0) {
        const int at = n + __popcll(b & ((1ull << lane) - 1));
        list[at] = (uint16_t)(s0 + lane);
        experts[at] = (uint16_t)slots[s0 + lane].expert;
        counts[at] = (uint16_t)c;
      }
      n += __popcll(b);
    }
    if (lane == 0) live = n;
    // a slot's chunks of 16 tokens, one turn each
    int at = 0;
    for (int k0 = 0; k0 < n; k0 += 64) {
      const int k = k0 + lane, c = k < n ? (counts[k] + kChunk - 1) / kChunk : 0;
      int before = c;  // inclusive sum over the lanes
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(before, off, 64);
        if (lane >= off) before += o;
      }
      for (int i = 0; i < c; ++i) turn[at + before - c + i] = (uint16_t)(4 * k + i);
      at += __shfl(before, 63, 64);
    }
    if (lane == 0) turns = at;
  }
  for (int o = threadIdx.x; o < kDownWaves * kRows * (kChunk + 1); o += kDownWaves * 64) (&sums[0][0][0])[o] = 0.0f;
  __syncthreads();
  const int nblk = I / kMxBlock, supers = (I + 511) / 512;
  const int slots_live = __builtin_amdgcn_readfirstlane(live);
  const int units = __builtin_amdgcn_readfirstlane(turns) * supers;
  const int n0 = (int)blockIdx.x * 16;
  uint8_t* const stage = stage_all[wave];
  // the wave's run of units: a turn's super-steps follow one another
  const int u0 = (int)((int64_t)units * wave / kDownWaves), u1 = (int)((int64_t)units * (wave + 1) / kDownWaves);
  auto load = [&](MxUnit& u, int i) {
    const int64_t row = (int64_t)__builtin_amdgcn_readfirstlane(experts[turn[i / supers] >> 2]) * H + n0;
    mx_load_unit(u, codes + row * nblk * 16, scales + row * nblk, 15, ((int64_t)E * H - row) * nblk, nblk, i % supers, lane);
  };
  float4_t acc = {};
  auto work = [&](const MxUnit& u, int i) {
    const int k4 = __builtin_amdgcn_readfirstlane(turn[i / supers]), k = k4 >> 2, c = k4 & 3, S = i % supers;
    const int sl = __builtin_amdgcn_readfirstlane(list[k]), count = __builtin_amdgcn_readfirstlane(counts[k]);
    const int64_t row = (int64_t)__builtin_amdgcn_readfirstlane(experts[k]) * H + n0;
    mx_stage_unit(u, stage, 15, ((int64_t)E * H - row) * nblk, nblk, S, lane);
    const int sc = mx_staged_scale(stage, lane);
    const int left = count - c * kChunk;  // rows past the last repeat it: their sums are not taken
    const MxPlace place = mx_place(0, (lane & 48) + ((lane & 15) < left ? lane & 15 : left - 1));
    mx_each_step([&](auto sel) {
      constexpr int s = decltype(sel)::value;
      MxActivations a;
      const int64_t f = (((int64_t)sl * chunks + c) * supers + S) * 4 + s;
      mx_load_activations(a, hp + f * kMxFragBytes, reinterpret_cast<const uint8_t*>(hs) + f * kMxFragScaleBytes, place);
      mx_multiply<s>(acc, a, mx_staged_weights(stage, s, lane), sc);
    });
    if (S == supers - 1 || i + 1 == u1) {  // the wave is through with the turn
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 4 * (lane >> 4) + e;
        if (r < left) sums[wave][slots[sl].token[c * kChunk + r]][lane & 15] += acc[e];
      }
      acc = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
  };
  MxUnit a, b;
  if (u0 < u1) load(a, u0);
  if (u0 + 1 < u1) load(b, u0 + 1);
  for (int i = u0; i < u1; i += 2) {
    work(a, i);
    if (i + 2 < u1) load(a, i + 2);
    if (i + 1 < u1) work(b, i + 1);
    if (i + 3 < u1) load(b, i + 3);
  }
  // the sum of a token's weights, slots in order
  if ((int)threadIdx.x < kRows) total[threadIdx.x] = 0.0f;
  __syncthreads();
  if (wave == 0) {
    for (int k = 0; k < slots_live; ++k) {
      const Slot& s = slots[list[k]];
      if (lane < s.count) total[s.token[lane]] += s.w[lane];
    }
  }
  __syncthreads();
  for (int o = threadIdx.x; o < T * kChunk; o += kDownWaves * 64) {
    const int t = o / kChunk, n = o % kChunk;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kDownWaves; ++w) v += sums[w][t][n];
    Y[(int64_t)t * H + n0 + n] = YT::from_f32(v / total[t]);
  }
}

struct Layout {
  int64_t chunks, slots, xfrags, hfrags;
  size_t logits, records, xp, xs, hp, hs, bytes;
};
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
Layout layout(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k) {
  Layout l;
  l.chunks = T <= 16 ? 1 : (T <= 32 ? 2 : 4);
  l.slots = T * top_k < E ? T * top_k : E;
  l.xfrags = l.chunks * ((H + 511) / 512 * 4);
  l.hfrags = l.slots * l.chunks * ((I + 511) / 512 * 4);
  l.logits = 0;
  l.records = l.logits + (size_t)E * kMaxTokens * 4;
  l.xp = up256(l.records + (size_t)l.slots * sizeof(Slot));
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
  Slot* const slots = reinterpret_cast<Slot*>(ws + l.records);
  uint32_t* const xs = reinterpret_cast<uint32_t*>(ws + l.xs);
  uint32_t* const hs = reinterpret_cast<uint32_t*>(ws + l.hs);
  const int groups = (T + kRouteTokens - 1) / kRouteTokens;
  const int blocks = T * kSuper * ((H + 511) / 512);
  moe_route_kernel<XT><<<(unsigned)(groups * E + (blocks + kRouteThreads - 1) / kRouteThreads), kRouteThreads, 0, stream>>>(
      X, router, T, H, E, groups, logits, ws + l.xp, xs);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  moe_up_kernel<<<dim3((unsigned)(I / kMxBlock), (unsigned)l.slots), kUpWaves * 64, 0, stream>>>(
      ws + l.xp, xs, up_codes, up_scales, logits, T, H, I, E, top_k, T * top_k < E ? 1 : 0, TC, slots, ws + l.hp, hs);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  moe_down_kernel<XT, TC><<<(unsigned)(H / 16), kDownWaves * 64, 0, stream>>>(ws + l.hp, hs, down_codes, down_scales,
                                                                             slots, (int)l.slots, T, H, I, E, Y);
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
    return l.chunks == 1   ? run(tag, std::integral_constant<int, 1>{})
           : l.chunks == 2 ? run(tag, std::integral_constant<int, 2>{})
                           : run(tag, std::integral_constant<int, 4>{});
  };
  return xdtype == 0 ? chunks(F16{}) : chunks(BF16{});
}

}  // namespace woq
