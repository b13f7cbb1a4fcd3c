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
// Launches:
//   route    logits, one workgroup per expert and 8 tokens
//   choose   one workgroup: the tokens' experts and shares, and the list of turns
//            (an expert and up to 16 of its tokens, in ascending order)
//   up       32 columns of h a time: gate and up rows, then p silu(g) u.  The share is
//            folded in here, where the values are still fp32; they are kept as two
//            bf16 numbers each (off by at most 2^-18 of the value, where fp32 would
//            need three and the registers hold two).
//   down     64 columns of a turn's products a time
//   combine  y from its experts' products, added in the order of choice (no atomics)
// A small layer of few tokens has no combine: its down adds over the experts itself.
// One token needs no list either: up and down work the choices out from the logits.
//
// bf16, H = 4096, I = 2048, 32 experts, 4 a token: 64 tokens 115 us, of which up 72
// (285 MB of weights, 4.0 TB/s) and down 36 (142 MB, 3.9 TB/s); one token 24 us, up
// 13.6, down 9.1, logits 4.5.  Before, a workgroup per 32 columns and turn (up) and per
// 16 columns of y over all turns (down) read the activations again for every 64 (16)
// weight rows, and its first loads had nothing before them to hide behind: 24 and 21 us
// more.
#include <cstddef>

#include "mxfp4_stream.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kChunk = 16;
constexpr int kMaxTokens = 64;
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 64;
constexpr int kRouteThreads = 512;
constexpr int kRouteTokens = 8;   // tokens per workgroup of the logits
constexpr int kChooseWaves = 16;
constexpr int kExpertWaves = 8;     // at most

// An expert and up to 16 of its tokens.
struct Turn {
  int expert, count;
  float share[kChunk];
  uint8_t token[kChunk];
};
struct Plan {
  int turns;
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

// logits [64][E]; a workgroup an expert and TOKENS tokens.
template <class XT, int TOKENS>
__global__ __launch_bounds__(kRouteThreads) void moe_route_kernel(const uint16_t* __restrict__ X,
                                                                  const uint16_t* __restrict__ router, int T, int H,
                                                                  int E, int groups, float* __restrict__ logits) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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

// A token's choices, one a lane: the wave works them out from its logits, lane
// holding those of the experts 64 j + lane.
struct Choice {
  int expert;
  float share;
};
template <int NJ>
__device__ inline Choice choose(const float (&logit)[NJ], int E, int top_k, int lane) {
  uint32_t key[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) key[j] = 64 * j + lane < E ? order_key(logit[j]) : 0u;
  uint32_t taken = 0;  // bit j: expert 64 j + lane
  int expert = 0;
  uint32_t chosen = 0, first = 0;
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
    if (c == 0) first = m;
    if (lane == c) {
      expert = id;
      chosen = m;
    }
  }
  const float w = lane < top_k ? expf(key_value(chosen) - key_value(first)) : 0.0f;
  return Choice{expert, w / team_sum(w, 64)};
}
// The same for two tokens of up to 32 experts, one in each half of the wave: lane
// holds the logit of expert lane % 32, and gets choice lane % 32.
__device__ inline Choice choose_pair(float logit, int E, int top_k, int lane) {
  const int l = lane & 31;
  const bool upper = lane >= 32;
  const uint32_t key = l < E ? order_key(logit) : 0u;
  bool taken = l >= E;
  int expert = 0;
  uint32_t chosen = 0, first = 0;
  for (int c = 0; c < top_k; ++c) {
    uint32_t v = taken ? 0u : key;
    auto step = [&](auto ctrl, auto rows) {
      const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
      v = v > o ? v : o;
    };
    step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xF>{});  // row_shr 1, 2, 4, 8
    step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xF>{});
    step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xF>{});
    step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xF>{});
    step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});  // row_bcast 15: lanes 31 and 63
    const uint32_t m0 = (uint32_t)__builtin_amdgcn_readlane((int)v, 31), m1 = (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
    const uint32_t m = upper ? m1 : m0;
    const uint64_t b = __ballot(!taken && key == m);
    const int i0 = __builtin_ctz((uint32_t)b), i1 = __builtin_ctz((uint32_t)(b >> 32));  // the lowest index of that key
    const int id = upper ? i1 : i0;
    taken |= l == id;
    first = c == 0 ? m : first;
    expert = l == c ? id : expert;
    chosen = l == c ? m : chosen;
  }
  const float w = l < top_k ? expf(key_value(chosen) - key_value(first)) : 0.0f;
  return Choice{expert, w / team_sum(w, 32)};
}
template <int NJ>
__device__ inline void load_logits(float (&logit)[NJ], const float* __restrict__ logits, int E, int lane) {
#pragma unroll
  for (int j = 0; j < NJ; ++j) logit[j] = 64 * j + lane < E ? logits[64 * j + lane] : 0.0f;
}

// One workgroup.  logits [T][E] -> the plan, its turns, and the row of the turns'
// products for each token's choices.
// NJ: lanes' experts, 64 NJ >= E; 0: two tokens a wave, E <= 32.
template <int NJ>
__global__ __launch_bounds__(kChooseWaves * 64) void moe_choose_kernel(const float* __restrict__ logits, int T, int E,
                                                                       int top_k, Plan* __restrict__ plan,
                                                                       Turn* __restrict__ turns,
                                                                       int* __restrict__ where) {
  __shared__ uint16_t ids[kMaxTokens * kMaxTopK];      // [token][choice]
  __shared__ float shares[kMaxTokens * kMaxTopK];
  __shared__ unsigned long long tokens[kMaxExperts];   // of an expert
  __shared__ uint16_t base[kMaxExperts];               // its first turn
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int e = threadIdx.x; e < E; e += kChooseWaves * 64) tokens[e] = 0;
  __syncthreads();
  auto note = [&](int t, int c, const Choice& choice) {
    ids[t * top_k + c] = (uint16_t)choice.expert;
    shares[t * top_k + c] = choice.share;
    atomicOr(&tokens[choice.expert], 1ull << t);
  };
  constexpr int kTokens = kMaxTokens / kChooseWaves;  // of a wave, at most
  if constexpr (NJ == 0) {
    float logit[kTokens / 2];
#pragma unroll
    for (int i = 0; i < kTokens / 2; ++i) {
      const int t = 2 * (wave + kChooseWaves * i) + (lane >> 5);
      logit[i] = t < T && (lane & 31) < E ? logits[t * E + (lane & 31)] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kTokens / 2; ++i) {
      const int t = 2 * (wave + kChooseWaves * i);
      if (t >= T) break;
      const Choice c = choose_pair(logit[i], E, top_k, lane);
      if (t + (lane >> 5) < T && (lane & 31) < top_k) note(t + (lane >> 5), lane & 31, c);
    }
  } else {
    float logit[kTokens][NJ];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const int t = wave + kChooseWaves * i;
      load_logits(logit[i], logits + (int64_t)(t < T ? t : 0) * E, E, lane);
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const int t = wave + kChooseWaves * i;
      if (t >= T) break;
      const Choice c = choose(logit[i], E, top_k, lane);
      if (lane < top_k) note(t, lane, c);
    }
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
    where[i] = (int)base[e] * kChunk + row;
  }
}

// Two numbers bf16 that hold v to within 2^-18 of itself: hi the nearest (the next
// one inside where that is not finite), lo the nearest to the rest.
struct Halves {
  uint16_t hi, lo;
};
__device__ inline Halves halves(float v) {
  const uint32_t bits = __builtin_bit_cast(uint32_t, v);
  uint16_t hi = BF16::from_f32(v);
  if ((hi & 0x7FFFu) == 0x7F80u) hi = (uint16_t)(bits >> 16);
  const bool finite = (bits & 0x7F800000u) != 0x7F800000u;
  return Halves{hi, finite ? BF16::from_f32(v - BF16::to_f32(hi)) : (uint16_t)0};
}

// h, p folded in, for down: of each turn and super-step four fragments
// (mxfp4_device.h) of the 16 tokens' hi, then four of their lo.  Up to 8 tokens are
// multiplied in one matrix step, their hi as the rows 0 .. 7 and their lo as the rows
// 8 .. 15, which join_halves adds; more in two steps.  Either way a unit's products
// with hi and with lo are sums of their own, added once: a token's bits do not depend
// on how many others share its turn.
constexpr int kHalfTokens = 8;
__host__ __device__ inline int64_t h_fragment(int64_t turn, int supers, int S) { return (turn * supers + S) * 8; }
// A lane's place in the fragments of hi: its token (rows past the turn's last one
// repeat it) and, of up to 8 tokens (first: of the group of 8), its half.
__device__ inline uint32_t h_place(int count, int lane) {
  const int r = lane & 15;
  return (uint32_t)(16 * ((lane & 48) + (r < count ? r : count - 1)));
}
__device__ inline uint32_t h_place_halves(int first, int count, int lane) {
  const int t = first + (lane & 7);
  return (uint32_t)(16 * ((lane & 48) + (t < count ? t : count - 1)) + (lane & 8 ? 4 * kMxFragBytes : 0));
}
// The products of a group of 8 tokens and of the next one -> rows 0 .. 15.
__device__ inline float4_t join_halves(float4_t a, float4_t b, int lane) {
  float4_t v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = (lane < 32 ? a[e] : b[e]) + __shfl_xor(lane < 32 ? b[e] : a[e], 32, 64);
  return v;
}

// The experts' products.  Item: a turn and 64 weight rows of its expert: UP, 32
// gate rows and their 32 up rows, which make 32 columns of h; else 64 rows of
// down, 64 columns of y.  A workgroup takes a run of items, K split between its
// waves (wave w: super-steps w, w + waves, ...).  The activations stay in
// registers while the turn does not change, and the next item's weights are on
// their way while an item's sums meet in LDS.
// NJ > 0: one token; every wave works its choices out from the logits, and turn k
// is choice k.  XT: of the activations; BF16 for h.
template <bool UP, int WAVES, int NJ, class XT>
__global__ __launch_bounds__(WAVES * 64, 2) void moe_experts_kernel(
    const uint16_t* __restrict__ X, const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
    const float* __restrict__ logits, int top_k, const Plan* __restrict__ plan, const Turn* __restrict__ turns, int K,
    int rows, int E, int groups, uint8_t* __restrict__ h, float* __restrict__ products) {
  constexpr int NT = 4;  // tiles of 16 rows; UP: gate rows, up rows, gate rows, up rows
  __shared__ __attribute__((aligned(16))) uint8_t stage_all[WAVES][kUnitStage];
  __shared__ float4_t parts[2][WAVES][NT][64];  // alternating: one barrier an item
  __shared__ float hbuf[kChunk + 1][kMxBlock + 1];  // the last row: zeros

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int nblk = K / kMxBlock, supers = (K + 511) / 512;
  __shared__ Choice choices[NJ > 0 ? WAVES : 1][NJ > 0 ? kMaxTopK : 1];
  if constexpr (NJ > 0) {
    float logit[NJ];
    load_logits(logit, logits, E, lane);
    choices[wave][lane] = choose(logit, E, top_k, lane);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  const int64_t items = (int64_t)(NJ > 0 ? top_k : plan->turns) * groups;
  const int i0 = (int)(items * blockIdx.x / gridDim.x), i1 = (int)(items * (blockIdx.x + 1) / gridDim.x);
  if (i0 >= i1) return;
  uint8_t* const stage = stage_all[wave];
  const int64_t all = (int64_t)E * rows;
  auto first_row = [&](int item) {
    const int k = item / groups;
    const int e = NJ > 0 ? __builtin_amdgcn_readfirstlane(choices[wave][k].expert) : turns[k].expert;
    return (int64_t)e * rows + item % groups * (UP ? 32 : 64);
  };
  // a turn's record, a dword a lane; on its way before the weights of its first item
  static_assert(sizeof(Turn) == 4 * 22 && offsetof(Turn, share) == 8 && offsetof(Turn, token) == 72, "read as dwords");
  auto record = [&](int k) {
    int l = lane;
    asm volatile("" : "+v"(l));  // addresses are worked out each time: kept, they spill
    return reinterpret_cast<const uint32_t*>(turns + k)[(uint32_t)(l < 22 ? l : 21)];
  };
  // rows past the expert's last (its columns are a multiple of 32) repeat the first tile
  auto tile_row = [&](int j, int item) {
    return UP ? (j & 1) * (rows / 2) + (j >> 1) * 16 : (item % groups * 64 + 16 * j < rows ? 16 * j : 0);
  };

  // the wave's next step, whose units are loaded as the current one's are used
  int item_n = i0, S_n = wave;
  uint32_t rec_n = NJ > 0 ? 0u : record(i0 / groups);
  int64_t row_n = first_row(i0);
  MxUnit u[NT];
  auto ahead = [&](int j, int l) {
    const int64_t row = row_n + tile_row(j, item_n);
    __builtin_amdgcn_sched_barrier(0);
    mx_load_unit(u[j], codes + row * nblk * 16, scales + row * nblk, 15, (all - row) * nblk, nblk, S_n, l);
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int j = 0; j < NT; ++j) ahead(j, lane);

  if (threadIdx.x < kMxBlock) hbuf[kChunk][threadIdx.x] = 0.0f;
  MxActivations a, lo;
  int turn = -1, count = 0, token = 0;
  float share = 0.0f;  // of row lane % 16; rows past the turn's last token repeat it
  for (int item = i0; item < i1; ++item) {
    const int k = item / groups, group = item % groups;
    const bool changed = k != turn;
    if (changed) {
      turn = k;
      if constexpr (NJ > 0) {
        count = 1;
        share = choices[wave][k].share;
      } else {
        count = __builtin_amdgcn_readlane((int)rec_n, 1);
        const int m = (lane & 15) < count ? lane & 15 : count - 1;
        share = __builtin_bit_cast(float, __shfl((int)rec_n, 2 + m, 64));
        token = UP ? __shfl((int)rec_n, 18 + m / 4, 64) >> (8 * (m & 3)) & 0xFF : 0;
      }
    }
    const bool two = !UP && count > kHalfTokens;  // matrix steps
    float4_t acc[NT] = {};  // UP; down adds its super-steps' products in LDS, which leaves registers for lo
    float4_t(*const part)[NT][64] = parts[(item - i0) & 1];
    const int64_t row0 = row_n;
    for (int S = wave; S < supers; S += waves) {
      if (changed || supers > waves) {
        int l = lane;
        asm volatile("" : "+v"(l));  // as above
        if constexpr (UP) {
          mx_load_activations(a, X + (int64_t)token * K, nblk, S, l);
          mx_mask_activations(a, nblk, S, l);
        } else {
          const uint8_t* const f = h + h_fragment(k, supers, S) * kMxFragBytes;
          mx_load_fragments(a, f, two ? h_place(count, l) : h_place_halves(0, count, l));
          if (two) mx_load_fragments(lo, f + 4 * kMxFragBytes, h_place(count, l));
        }
      }
      S_n = S + waves;
      if (S_n >= supers) {
        S_n = wave;
        if (++item_n < i1) {
          if (NJ == 0 && item_n / groups != k) rec_n = record(item_n / groups);
          row_n = first_row(item_n);
        }
      }
      auto multiply = [&](auto more) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          int l = lane;
          asm volatile("" : "+v"(l));  // as above
          mx_stage_unit(u[j], stage, 15, (all - (row0 + tile_row(j, item))) * nblk, nblk, S, l);
          if constexpr (decltype(more)::value) ahead(j, l);
          if constexpr (UP) {
            mx_multiply_unit<XT>(acc[j], a, stage, l);
          } else {
            float4_t v = {};
            if (two) {
              float4_t w = {};
              mx_multiply_unit<XT, true>(v, a, w, lo, stage, l);
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] += w[e];
            } else {
              mx_multiply_unit<XT>(v, a, stage, l);
              v = join_halves(v, float4_t{}, l);
            }
            float4_t& sum = part[wave][j][l];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += S == wave ? 0.0f : sum[e];
            sum = v;
          }
        }
      };
      if (item_n < i1)
        multiply(std::true_type{});
      else
        multiply(std::false_type{});
    }
    int l = lane;
    asm volatile("" : "+v"(l));  // as above
    if constexpr (UP)
#pragma unroll
      for (int j = 0; j < NT; ++j) part[wave][j][l] = acc[j];
    __syncthreads();
    // value (row m, tile j, column c) of a wave: part[w][j][(m / 4) 16 + c][m % 4]
    auto sum = [&](int m, int j, int c) {
      float p[WAVES], v = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) p[w] = part[w][j][(m >> 2) * 16 + c][m & 3];
#pragma unroll
      for (int w = 0; w < WAVES; ++w) v += w < waves ? p[w] : 0.0f;
      return v * kMxGain<XT>;
    };
    if constexpr (UP) {
      // wave w takes the rows 2 w, 2 w + 1, + 2 waves, ...
      for (int m0 = 2 * wave; m0 < count; m0 += 2 * waves) {
        const int m = m0 + (l >> 5), c = l & 31;
        if (m < count) {
          const float g = sum(m, (c >> 4) * 2, c & 15), v = sum(m, (c >> 4) * 2 + 1, c & 15);
          hbuf[m][c] = g / (1.0f + expf(-g)) * v;
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      // a lane writes a row's block; behind the last block of h the rest of its
      // super-step is zeros
      const int m = l & 15, hsupers = (groups + kSuper - 1) / kSuper;
      const int end = group == groups - 1 ? kSuper * hsupers : group + 1;
      if (m < count && (m >> 1) % waves == wave) {
        for (int b = group + (l >> 4); b < end; b += 4) {
          const float* const row = hbuf[b == group ? m : kChunk];
          const float scale = b == group ? share : 0.0f;
          uint8_t* const to = h + (h_fragment(k, hsupers, b / kSuper) + b % 4) * kMxFragBytes + 16 * ((b % kSuper / 4) * kChunk + m);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            u32x4_t hi = {}, lo = {};
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const Halves v = halves(scale * row[8 * q + c]);
              hi[c / 2] |= (uint32_t)v.hi << (16 * (c % 2));
              lo[c / 2] |= (uint32_t)v.lo << (16 * (c % 2));
            }
            *reinterpret_cast<u32x4_t*>(to + 1024 * q) = hi;
            *reinterpret_cast<u32x4_t*>(to + 4 * kMxFragBytes + 1024 * q) = lo;
          }
        }
      }
    } else {
      const int n = group * 64 + l;
      for (int m = wave; m < count; m += waves)
        if (n < rows) (products + (int64_t)k * kChunk * rows)[(uint32_t)(m * rows + n)] = sum(m, l >> 4, l & 15);
    }
  }
}

// Few units of weights: columns [16 b, 16 b + 16) of y for up to 16 tokens, over all
// turns' super-steps, which the waves share out two at a time.  A unit's products meet
// in LDS; a token's are added in its order of choice, a choice's super-steps in theirs,
// so that they do not depend on the other tokens.  NJ as above: then the units are in
// that order themselves, and go in rounds.
constexpr int kDirectUnits = 36, kRoundUnits = 64;
template <class YT, int NJ>
__global__ __launch_bounds__(kExpertWaves * 64) void moe_direct_down_kernel(
    const uint8_t* __restrict__ h, const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
    const float* __restrict__ logits, int top_k, const Plan* __restrict__ plan, const Turn* __restrict__ turns,
    const int* __restrict__ where, int T, int H, int I, int E, uint16_t* __restrict__ Y) {
  constexpr int W = kExpertWaves, kRows = NJ > 0 ? 1 : kChunk, kUnits = NJ > 0 ? kRoundUnits : kDirectUnits;
  __shared__ __attribute__((aligned(16))) uint8_t stage_all[W][kUnitStage];
  __shared__ float parts[kUnits][kRows][kChunk + 1];
  __shared__ int rows[NJ > 0 ? 1 : kChunk * kMaxTopK];  // of the tokens' choices, [token][choice]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nblk = I / kMxBlock, supers = (I + 511) / 512;
  const int n0 = (int)blockIdx.x * 16;
  uint8_t* const stage = stage_all[wave];
  Choice choice = {};
  if constexpr (NJ > 0) {
    float logit[NJ];
    load_logits(logit, logits, E, lane);
    choice = choose(logit, E, top_k, lane);
  } else {
    for (int i = threadIdx.x; i < T * top_k; i += W * 64) rows[i] = where[i];
  }
  const int units = (NJ > 0 ? top_k : plan->turns) * supers;
  struct Work {
    MxUnit u;
    MxActivations a;
  };
  auto row_of = [&](int i) {
    const int k = i / supers;
    const int e = NJ > 0 ? __builtin_amdgcn_readlane(choice.expert, k) : turns[k].expert;
    return (int64_t)e * H + n0;
  };
  auto count_of = [&](int i) { return NJ > 0 ? 1 : turns[i / supers].count; };
  auto activations = [&](MxActivations& a, int i, int first) {
    mx_load_fragments(a, h + h_fragment(i / supers, supers, i % supers) * kMxFragBytes, h_place_halves(first, count_of(i), lane));
  };
  auto load = [&](Work& w, int i) {
    const int64_t row = row_of(i);
    mx_load_unit(w.u, codes + row * nblk * 16, scales + row * nblk, 15, ((int64_t)E * H - row) * nblk, nblk, i % supers, lane);
    activations(w.a, i, 0);
  };
  auto work = [&](Work& w, int i) {
    float4_t acc = {}, more = {};
    mx_stage_unit(w.u, stage, 15, ((int64_t)E * H - row_of(i)) * nblk, nblk, i % supers, lane);
    mx_multiply_unit<BF16>(acc, w.a, stage, lane);
    const int count = count_of(i);
    if (NJ == 0 && count > kHalfTokens) {
      activations(w.a, i, kHalfTokens);
      mx_multiply_unit<BF16>(more, w.a, stage, lane);
    }
    acc = join_halves(acc, more, lane);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (4 * (lane >> 4) + e < count) parts[i % kUnits][NJ > 0 ? 0 : 4 * (lane >> 4) + e][lane & 15] = acc[e];
  };
  float v = 0.0f, p = 0.0f;  // NJ: of thread n's column, and of the choice that a round may cut
  int left = supers;
  for (int i0 = 0; i0 < units; i0 += kUnits) {
    const int i1 = i0 + kUnits < units ? i0 + kUnits : units;
    // an odd last unit is loaded twice and multiplied once
    for (int i = i0 + wave; i < i1; i += 2 * W) {
      const bool two = i + W < i1;
      Work a, b;
      load(a, i);
      load(b, two ? i + W : i);
      __builtin_amdgcn_sched_barrier(0);  // all loads start before the first product
      work(a, i);
      if (two) work(b, i + W);
    }
    __syncthreads();
    if constexpr (NJ > 0) {
      if ((int)threadIdx.x < kChunk)
#pragma unroll 8
        for (int i = 0; i < i1 - i0; ++i) {
          p += parts[i][0][threadIdx.x];
          const bool last = --left == 0;  // of a choice
          v += last ? p : 0.0f;
          p = last ? 0.0f : p;
          left = last ? supers : left;
        }
      if (i1 < units) __syncthreads();
    }
  }
  if ((int)threadIdx.x < T * kChunk) {
    const int t = threadIdx.x / kChunk, n = threadIdx.x % kChunk;
    if constexpr (NJ == 0)
      for (int c = 0; c < top_k; ++c) {
        const int row = rows[t * top_k + c];
        p = 0.0f;
        for (int S = 0; S < supers; ++S) p += parts[row / kChunk * supers + S][row % kChunk][n];
        v += p;
      }
    Y[(int64_t)t * H + n0 + n] = YT::from_f32(v * kMxGain<BF16>);
  }
}

// y[t] = the sum of its experts' rows of `products`, in the order of choice.
template <class YT>
__global__ __launch_bounds__(64) void moe_combine_kernel(const float* __restrict__ products, const int* __restrict__ where,
                                                         int H, int top_k, uint16_t* __restrict__ Y) {
  const int n = ((int)blockIdx.x * 64 + (int)threadIdx.x) * 4, t = blockIdx.y;
  if (n >= H) return;
  float4_t v = {};
  for (int c = 0; c < top_k; ++c) {
    const float4_t p = *reinterpret_cast<const float4_t*>(products + (int64_t)where[t * top_k + c] * H + n);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += p[e];
  }
  const uint32_t lo = (uint32_t)YT::from_f32(v[0]) | (uint32_t)YT::from_f32(v[1]) << 16;
  const uint32_t hi = (uint32_t)YT::from_f32(v[2]) | (uint32_t)YT::from_f32(v[3]) << 16;
  *reinterpret_cast<u32x2_t*>(Y + (int64_t)t * H + n) = u32x2_t{lo, hi};
}

struct Layout {
  int64_t turns;
  size_t logits, plan, records, where, h, products, bytes;
};
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
Layout layout(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k) {
  Layout l;
  // a turn for each chosen expert and one for each further 16 tokens of it
  l.turns = (T * top_k < E ? T * top_k : E) + T * top_k / kChunk;
  l.logits = 0;
  l.plan = up256((size_t)E * T * 4);
  l.records = l.plan + 256;
  l.where = up256(l.records + (size_t)l.turns * sizeof(Turn));
  l.h = up256(l.where + (size_t)(T * top_k) * 4);
  l.products = l.h + (size_t)h_fragment(l.turns, (int)((I + 511) / 512), 0) * kMxFragBytes;
  l.bytes = l.products + (size_t)(l.turns * kChunk * H) * 4;
  return l;
}

template <class XT>
hipError_t launch(const uint16_t* X, const uint16_t* router, const uint8_t* up_codes, const uint8_t* up_scales,
                  const uint8_t* down_codes, const uint8_t* down_scales, int T, int H, int I, int E, int top_k,
                  uint16_t* Y, uint8_t* ws, const Layout& l, hipStream_t stream) {
  float* const logits = reinterpret_cast<float*>(ws + l.logits);
  Plan* const plan = reinterpret_cast<Plan*>(ws + l.plan);
  Turn* const turns = reinterpret_cast<Turn*>(ws + l.records);
  int* const where = reinterpret_cast<int*>(ws + l.where);
  float* const products = reinterpret_cast<float*>(ws + l.products);
  uint8_t* const h = ws + l.h;
  const int tokens = T == 1 ? 1 : kRouteTokens;
  const int groups = (T + tokens - 1) / tokens;
  const unsigned grid = (unsigned)(groups * E);
  if (T == 1)
    moe_route_kernel<XT, 1><<<grid, kRouteThreads, 0, stream>>>(X, router, T, H, E, groups, logits);
  else
    moe_route_kernel<XT, kRouteTokens><<<grid, kRouteThreads, 0, stream>>>(X, router, T, H, E, groups, logits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int kLarge = kMaxExperts / 64;
  if (T > 1) {
    // (64 tokens of 32 experts, four each: 5.2 us two to a wave, 8.0 one by one)
    auto* const f = E <= 32 ? moe_choose_kernel<0> : (E <= 64 ? moe_choose_kernel<1> : moe_choose_kernel<kLarge>);
    f<<<1, kChooseWaves * 64, 0, stream>>>(logits, T, E, top_k, plan, turns, where);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // a wave for every super-step of a row, up to 8; 8 waves fill a compute unit
  auto experts = [&](auto up, auto nj, const uint8_t* codes, const uint8_t* scales, int K, int rows, int groups) {
    constexpr bool kUp = decltype(up)::value;
    constexpr int kNj = decltype(nj)::value;
    using AT = std::conditional_t<kUp, XT, BF16>;
    const int supers = (K + 511) / 512, waves = supers < kExpertWaves ? supers : kExpertWaves;
    auto* const f = waves > 4 ? moe_experts_kernel<kUp, kExpertWaves, kNj, AT> : moe_experts_kernel<kUp, 4, kNj, AT>;
    f<<<256u * (unsigned)(kExpertWaves / waves), (unsigned)(waves * 64), 0, stream>>>(X, codes, scales, logits, top_k, plan, turns,
                                                                                      K, rows, E, groups, h, products);
    return hipGetLastError();
  };
  auto up = [&](auto nj) { return experts(std::true_type{}, nj, up_codes, up_scales, H, 2 * I, I / kMxBlock); };
  // Few units of down's weights go straight to y.  Whole layers of T x H x I, us, direct /
  // in two launches, by turns (at most) x super-steps:
  //   4    2 x 1024 x 512    25 / 26        20  16 x 4096 x 1024   32 / 40
  //   10   3 x 4096 x 1024   28 / 35        32   2 x 4096 x 2048   42 / 43
  //   16   4 x 2048 x 512    27 / 41        34  16 x 2048 x 512    31 / 36
  //   17   8 x 1024 x 512    26 / 32        36  16 x 4096 x 512    44 / 53
  // More units' products would not leave two workgroups a compute unit their LDS; with
  // sums of another order, 68 (8 x 2048 x 768) took 40 / 37 and 93 (5 x 2080 x 1056) 61 / 49.
  const bool direct = T == 1 || (T <= kChunk && l.turns * ((I + 511) / 512) <= kDirectUnits);
  using Nj0 = std::integral_constant<int, 0>;
  using Nj1 = std::integral_constant<int, 1>;
  using NjN = std::integral_constant<int, kLarge>;
  e = T > 1 ? up(Nj0{}) : (E <= 64 ? up(Nj1{}) : up(NjN{}));
  if (e != hipSuccess) return e;
  if (direct) {
    auto* const f = T > 1 ? moe_direct_down_kernel<XT, 0> : (E <= 64 ? moe_direct_down_kernel<XT, 1> : moe_direct_down_kernel<XT, kLarge>);
    f<<<(unsigned)(H / 16), kExpertWaves * 64, 0, stream>>>(h, down_codes, down_scales, logits, top_k, plan, turns, where, T, H, I, E, Y);
    return hipGetLastError();
  }
  e = experts(std::false_type{}, Nj0{}, down_codes, down_scales, I, H, (H + 63) / 64);
  if (e != hipSuccess) return e;
  moe_combine_kernel<XT><<<dim3((unsigned)((H + 255) / 256), (unsigned)T), 64, 0, stream>>>(products, where, H, top_k, Y);
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
  auto run = [&](auto tag) {
    return launch<decltype(tag)>(
        static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(router), static_cast<const uint8_t*>(up_codes),
        static_cast<const uint8_t*>(up_scales), static_cast<const uint8_t*>(down_codes),
        static_cast<const uint8_t*>(down_scales), (int)T, (int)H, (int)I, (int)E, top_k, static_cast<uint16_t*>(Y),
        static_cast<uint8_t*>(workspace), l, stream);
  };
  return xdtype == 0 ? run(F16{}) : run(BF16{});
}

}  // namespace woq
