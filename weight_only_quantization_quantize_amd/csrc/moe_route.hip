// Routing to experts, and its gradient.  Of a token's logits x[e]:
//   s = softmax(x) or sigmoid(x)
//   order of the experts: by x, or, with a bias b, by s + b in 64 bits; the lower index first
//     among equals; -infinity (a masked expert) after every number, a NaN last
//   groups: E / groups neighbours each; only the top_groups of them with the largest sum of
//     their group_top best keys (x or s + b; of two without a bias: s) are chosen from
//   w = scale s, over the sum of the chosen experts' s where that is asked for
//
// Bound by vector instructions: a logit is 2 or 4 bytes, its score and its part in the
// choice 85 instructions (16384 tokens of 256 experts, 8 groups, a bias: 1370 a wave of 1024
// logits, four waves a SIMD, which issue one 60% of the time; 20.5 us).  So the usual routing (route_row) has four tokens a
// wave, 16 lanes each, neighbouring experts in a lane, and decides in 32 bits what they decide:
//   scores p = 1 / (1 + 2^(-x log2 e)) are off by at most 2^-21, 2^((x - max) log2 e) / sum
//   by 2^-19, s + b by 2^-24 of itself more;
//   a key is cut to make room for its expert's index in its low bits (8, or 9 from 257
//   experts on), so that keys are distinct, lanes sort theirs by a network of min and max,
//   and a round of choice is a maximum over 16 lanes;
//   where two neighbours among the chosen and the best one left out are too near to be told
//   apart, the exact keys (64 bits; the logits where there is no bias) of the chosen and the
//   two next put them in order, one a lane; no others can be meant as long as the third is
//   further away.  Groups too near to be told apart have their sums worked out in 64 bits.
// What is left (three near neighbours more, NaN, infinities) goes the exact way (route_token),
// a wave a token, as do more than 13 choices and groups that are not whole lanes of experts.
#include <utility>

#include "int8_device.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kWaves = 4;  // tokens of a workgroup

template <class XT>
__device__ inline float load_logit(const void* __restrict__ x, int64_t i) {
  if constexpr (kElementBytes<XT> == 4)
    return static_cast<const float*>(x)[i];
  else
    return XT::to_f32(static_cast<const uint16_t*>(x)[i]);
}

// A number's order as an unsigned one; the zeros are equal, a NaN comes below -infinity.
__device__ inline uint64_t order_key(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
  if ((b & 0x7FFFFFFFFFFFFFFFull) > 0x7FF0000000000000ull) return 1ull;
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
template <int TEAM = 64>
__device__ inline double wave_sum(double v) {
#pragma unroll
  for (int off = TEAM / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
__device__ inline uint64_t wave_max(uint64_t v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)v, off, 64);
    v = v > o ? v : o;
  }
  return v;
}
__device__ inline bool is_masked(float x) { return x == -__builtin_inff(); }
__device__ inline double sigmoid64(float x) { return 1.0 / (1.0 + exp(-(double)x)); }

// The weights of the chosen experts' logits, lane c of TEAM lanes holding the c-th (used: c <
// top_k); max, sum: of the row, as softmax without renormalisation needs them, or, where given
// says so, max of the chosen ones.
template <int TEAM = 64>
__device__ inline double weight_of(float x, bool used, bool sigmoid, bool renormalize, float max, double sum, bool given = false) {
  double s = 0.0;
  if (sigmoid) {
    if (used) s = sigmoid64(x);
  } else {
    if (renormalize) {  // the row's sum cancels
      if (!given) max = team_max(used ? x : -__builtin_inff(), TEAM);
      max = is_masked(max) ? 0.0f : max;
    }
    if (used) s = exp((double)x - (double)max);
  }
  if (renormalize) sum = wave_sum<TEAM>(s);
  if (sigmoid && !renormalize) return s;
  return sum == 0.0 ? 0.0 : s / sum;
}

// What a routing is asked for.
struct Routing {
  int E, top_k, sigmoid, groups, top_groups, group_top, renormalize;
  float scale;
};

// A token by a wave, in 64 bits; lane l holds the experts 64 j + l, 64 NJ >= E.  keys, ranks:
// LDS of the wave's own, 64 NJ numbers each.
template <class XT, int NJ>
__device__ __noinline__ void route_token(const void* __restrict__ logits, int64_t t, Routing r, const float* __restrict__ bias,
                                         double* keys, double* ranks, int32_t* __restrict__ experts,
                                         float* __restrict__ weights) {
  const int E = r.E, top_k = r.top_k, groups = r.groups, lane = threadIdx.x & 63;
  const bool sigmoid = r.sigmoid, renormalize = r.renormalize;
  float x[NJ], max = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    x[j] = 64 * j + lane < E ? load_logit<XT>(logits, t * E + 64 * j + lane) : -__builtin_inff();
    max = fmaxf(max, x[j]);
  }
  max = team_max(max, 64);
  max = is_masked(max) ? 0.0f : max;
  double s[NJ], sum = 0.0;
  const bool wide = bias || (groups > 1 && r.group_top > 1);  // scores of all experts
  if (wide || (!sigmoid && !renormalize)) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      s[j] = sigmoid ? sigmoid64(x[j]) : exp((double)x[j] - (double)max);
      sum += s[j];
    }
    sum = wave_sum(sum);
  }
  uint64_t key[NJ];  // 0: not to be chosen
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = 64 * j + lane;
    double k = x[j], by = x[j];
    if (wide) {
      const double p = sigmoid || sum == 0.0 ? s[j] : s[j] / sum;
      if (bias)
        by = k = is_masked(x[j]) ? (double)x[j] : p + (double)bias[e < E ? e : 0];
      else
        by = is_masked(x[j]) ? (double)x[j] : p;
    }
    key[j] = e < E ? order_key(k) : 0ull;
    if (groups > 1) keys[e] = by;
  }
  if (groups > 1) {
    // lane g: groups g, g + 64, ...
    const int per = E / groups;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    for (int g = lane; g < groups; g += 64) {
      double best = keys[g * per], next = -__builtin_inf();
      uint64_t kb = order_key(best), kn = 0ull;
      for (int i = 1; i < per; ++i) {
        const double v = keys[g * per + i];
        const uint64_t kv = order_key(v);
        if (kv > kb) {
          next = best, kn = kb;
          best = v, kb = kv;
        } else if (kv > kn) {
          next = v, kn = kv;
        }
      }
      ranks[g] = r.group_top > 1 ? best + next : best;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = 64 * j + lane, g = e < E ? e / per : 0;
      const uint64_t mine = order_key(ranks[g]);
      int before = 0;
      for (int i = 0; i < groups; ++i) {
        const uint64_t o = order_key(ranks[i]);
        before += o > mine || (o == mine && i < g);
      }
      if (before >= r.top_groups) key[j] = 0ull;
    }
  }
  float chosen = 0.0f;
  int expert = 0;
  for (int c = 0; c < top_k; ++c) {
    uint64_t m = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) m = key[j] > m ? key[j] : m;
    m = wave_max(m);
    int id = -1;  // the lowest index of that key
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (id < 0) {
        const uint64_t b = __ballot(key[j] == m);
        if (b) id = 64 * j + __builtin_ctzll(b);
      }
    float v = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (id >> 6 == j) {
        v = x[j];
        if ((id & 63) == lane) key[j] = 0ull;
      }
    v = __shfl(v, id & 63, 64);
    if (lane == c) {
      chosen = v;
      expert = id;
    }
  }
  const double w = weight_of(chosen, lane < top_k, sigmoid, renormalize, max, sum);
  if (lane < top_k) {
    experts[t * top_k + lane] = expert;
    weights[t * top_k + lane] = (float)(w * (double)r.scale);
  }
}

constexpr int kRow = 16;            // lanes of a token
constexpr int kRowTokens = 4;       // tokens of a wave
constexpr int kMore = 3;            // candidates beside the chosen

// A number's order as an unsigned one; the zeros are equal, a NaN comes below -infinity.
__device__ inline uint32_t order_key32(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  const uint32_t k = b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
  return v != v ? 0x10000u : k;
}
__device__ inline float key_value(uint32_t k) {  // of a NaN's, and of a cut -infinity's, a NaN
  return __builtin_bit_cast(float, (k >> 31) ? k & 0x7FFFFFFFu : ~k);
}
// f over the 16 lanes of a row, in all of them.
template <class T, class F>
__device__ inline T row_all(T v, F&& f) {
  auto step = [&](auto n) {
    constexpr int kRor = 0x120 + decltype(n)::value;
    const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kRor, 0xF, 0xF, false);
    v = f(v, __builtin_bit_cast(T, o));
  };
  step(std::integral_constant<int, 8>{});
  step(std::integral_constant<int, 4>{});
  step(std::integral_constant<int, 2>{});
  step(std::integral_constant<int, 1>{});
  return v;
}
// Keys of n elements in descending order, by Batcher's odd-even merge network.
template <int N>
struct Network {
  int count = 0;
  uint8_t a[N * 8] = {}, b[N * 8] = {};
  constexpr Network() {
    for (int p = 1; p < N; p *= 2)
      for (int k = p; k >= 1; k /= 2)
        for (int j = k % p; j + k < N; j += 2 * k)
          for (int i = 0; i < k && i + j + k < N; ++i)
            if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) a[count] = (uint8_t)(i + j), b[count++] = (uint8_t)(i + j + k);
  }
};
template <int N, int... I>
__device__ __forceinline__ void sort_descending(uint32_t (&v)[N], std::integer_sequence<int, I...>) {
  constexpr Network<N> net;
  auto exchange = [&](int i, int j) {
    const uint32_t x = v[i], y = v[j];
    v[i] = x > y ? x : y;
    v[j] = x > y ? y : x;
  };
  (exchange(net.a[I], net.b[I]), ...);
}
template <int N>
__device__ __forceinline__ void sort_descending(uint32_t (&v)[N]) {
  sort_descending(v, std::make_integer_sequence<int, Network<N>().count>{});
}

template <class T>
__device__ inline T row_rotated(T v, int n) {  // of the lane n further on
  return __shfl(v, ((int)threadIdx.x & 48) | (((int)threadIdx.x + n) & 15), 64);
}

// A lane's `own` elements from at on, of any alignment; -infinity behind them.
template <class XT, int NJ>
__device__ __forceinline__ void load_lane(float (&x)[NJ], const void* __restrict__ from, int64_t at, int own) {
  typedef typename Int8Out<XT>::type T;
  constexpr int kVector = kElementBytes<XT> == 4 || NJ < 8 ? 4 : 8;
#pragma unroll
  for (int j0 = 0; j0 < NJ; j0 += kVector) {
    if (j0 + kVector <= own) {
      T v[kVector];
      __builtin_memcpy(v, static_cast<const T*>(from) + at + j0, sizeof(v));
#pragma unroll
      for (int j = 0; j < kVector; ++j) x[j0 + j] = load_logit<XT>(v, j);
    } else if (j0 < own) {
#pragma unroll
      for (int j = j0; j < j0 + kVector; ++j) x[j] = load_logit<XT>(from, at + (j < own ? j : own - 1));
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) x[j] = j < own ? x[j] : -__builtin_inff();
}

// A logit's score in 64 bits (max, sum: a softmax's).
__device__ inline double score64(float x, bool sigmoid, float max, double sum) {
  return sigmoid ? sigmoid64(x) : exp((double)x - (double)max) / sum;
}
template <int NJ>
__device__ inline double softmax_sum(const float (&x)[NJ], float max) {
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) sum += exp((double)x[j] - (double)max);
  return wave_sum<kRow>(sum);
}

// Four tokens by a wave, lane l of a row of 16 the n = ceil(E / 16) experts from l n on, n <=
// NJ.  Returns whether the row's choice is decided; then it is written.
template <class XT, int NJ>
__device__ __forceinline__ bool route_row(const void* __restrict__ logits, int64_t t, const Routing& r,
                                          const float* __restrict__ bias, int32_t* __restrict__ experts,
                                          float* __restrict__ weights) {
  constexpr uint32_t kIndex = NJ > 16 ? 511u : 255u;
  const float kClose = r.sigmoid ? 0x1p-20f : 0x1p-18f;  // of two scores, and of 1 + |key|
  constexpr float kLog2e = 1.44269504088896341f;
  const int E = r.E, top_k = r.top_k, l = threadIdx.x & (kRow - 1), n = (E + kRow - 1) / kRow, e0 = l * n;
  const int own = E - e0 < n ? E - e0 : n;  // of the lane; the rest counts as masked
  const float inf = __builtin_inff();
  float x[NJ], max = -inf;
  load_lane<XT, NJ>(x, logits, t * E + e0, own);
  auto larger = [](float a, float b) { return fmaxf(a, b); };
  const bool all = !r.sigmoid && !r.renormalize;
  const bool scored = bias || (r.groups > 1 && r.group_top > 1);
  double sum = 0.0;
  if (!r.sigmoid && (scored || all)) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) max = fmaxf(max, x[j]);
    max = row_all(max, larger);
    max = is_masked(max) ? 0.0f : max;
  }
  if (all) sum = softmax_sum(x, max);
  float by[NJ];  // what groups are compared by
  uint32_t key[NJ];
  // (each uniform question is asked once, not for every expert: a branch and a wait each took
  // 16384 tokens of 256 experts 46 us)
  if (scored) {
    if (r.sigmoid) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) by[j] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x[j] * kLog2e));
    } else {
      float part = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        by[j] = __builtin_amdgcn_exp2f((x[j] - max) * kLog2e);
        part += by[j];
      }
      const float inverse = __builtin_amdgcn_rcpf(row_all(part, [](float a, float b) { return a + b; }));
#pragma unroll
      for (int j = 0; j < NJ; ++j) by[j] *= inverse;
    }
    if (bias) {
      float b[NJ];
      load_lane<F32, NJ>(b, bias, e0, own);
#pragma unroll
      for (int j = 0; j < NJ; ++j) by[j] += b[j];
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) by[j] = is_masked(x[j]) ? x[j] : by[j];
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) by[j] = x[j];
  }
  if (bias) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) key[j] = order_key32(by[j]);
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) key[j] = order_key32(x[j]);
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) key[j] = j < own ? key[j] : 0u;
  bool sure = true;
  if (r.groups > 1) {  // a group is kRow / groups lanes
    float best = -inf, next = -inf;
    bool odd = false;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      odd |= j < own && !(fabsf(by[j]) < inf) && !is_masked(x[j]);
      next = fmaxf(next, fminf(best, by[j]));
      best = fmaxf(best, by[j]);
    }
    const int lanes = kRow / r.groups;
    for (int off = 1; off < lanes; off <<= 1) {
      const float b = __shfl_xor(best, off, 64), n = __shfl_xor(next, off, 64);
      next = fmaxf(fminf(best, b), fmaxf(next, n));
      best = fmaxf(best, b);
    }
    const float rank = r.group_top > 1 ? best + next : best;
    // By how much the rank may be off: its scores' errors, and each key's and the sum's rounding, 2^-24 of the keys and not of
    // what is left of them where they cancel.  A best logit is exact, and so is -infinity of masked experts.
    const float size = r.group_top > 1 ? fabsf(best) + fabsf(next) : fabsf(best);
    const bool exact = !scored || is_masked(r.group_top > 1 ? next : best);
    const float off = exact ? 0.0f : kClose + 0x1p-22f * size;
    int before = 0;
#pragma unroll
    for (int n = 1; n < kRow; ++n) before += row_rotated(rank, n) > rank ? 1 : 0;
    bool kept = before < r.top_groups * lanes;
    // (sums past 32 bits' range are infinite, and so is what they may be off by: never told apart)
    const float high = off < inf ? rank + off : inf, low = off < inf ? rank - off : -inf;
    const float last = -row_all(kept ? -low : -inf, larger), first = row_all(kept ? -inf : high, larger);
    // (equal ranks are not told apart here)
    const int keeps = row_all(kept ? 1 : 0, [](int a, int b) { return a + b; });
    const bool told = r.top_groups == r.groups || (last > first && keeps == r.top_groups * lanes);
    if (__any(!told)) {  // the groups' sums in 64 bits
      const double total = scored && !r.sigmoid ? softmax_sum(x, max) : 1.0;
      double best = -inf, next = -inf;
#pragma unroll 1
      for (int j = 0; j < own; ++j) {
        const float y = load_logit<XT>(logits, t * E + e0 + j);
        double v = y;
        if (scored && !is_masked(y)) v = score64(y, r.sigmoid, max, total) + (bias ? (double)bias[e0 + j] : 0.0);
        next = fmax(next, fmin(best, v));
        best = fmax(best, v);
      }
      for (int off = 1; off < lanes; off <<= 1) {
        const double b = __shfl_xor(best, off, 64), n = __shfl_xor(next, off, 64);
        next = fmax(fmin(best, b), fmax(next, n));
        best = fmax(best, b);
      }
      const double mine = r.group_top > 1 ? best + next : best;
      int ahead = 0;
#pragma unroll 1
      for (int n = 1; n < kRow; ++n) {
        const double o = row_rotated(mine, n);
        ahead += o > mine || (o == mine && ((l + n) & (kRow - 1)) / lanes < l / lanes) ? 1 : 0;
      }
      kept = told ? kept : ahead < r.top_groups * lanes;
    }
    // NaN and infinities may have no order above
    sure = !row_all(odd ? 1 : 0, [](int a, int b) { return a | b; });
    if (!kept)
#pragma unroll
      for (int j = 0; j < NJ; ++j) key[j] = 0u;
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) key[j] = key[j] ? (key[j] & ~kIndex) | (kIndex - (uint32_t)(e0 + j)) : 0u;
  sort_descending(key);
  // choice c in lane c, and kMore more
  uint32_t choice = 0;
  for (int c = 0; c < top_k + kMore; ++c) {
    const uint32_t m = row_all(key[0], [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    const uint32_t mine = key[0] == m ? ~0u : 0u;  // (a mask: a choice of two places is not kept in registers)
#pragma unroll
    for (int j = 0; j < NJ; ++j) key[j] = (key[j] & ~mine) | ((j + 1 < NJ ? key[j + 1] : 0u) & mine);
    choice = l == c ? m : choice;
  }
  int expert = choice ? (int)(kIndex - (choice & kIndex)) : 0;
  // whether a comes before b whatever the cut and the scores' errors (16-bit logits are not cut)
  auto apart = [&](uint32_t a, uint32_t b) {
    if (b == 0u) return true;
    const uint32_t x = a & ~kIndex, y = b & ~kIndex;
    if (!bias) return kElementBytes<XT> == 2 || x != y;
    const float v = key_value(x), w = key_value(y), cut = (float)(kIndex + 1) * 0x1p-22f;
    return v - w > kClose * (1.0f + fabsf(w)) + cut * (fabsf(v) + fabsf(w));
  };
  // (read by all lanes: those of a branch not taken give 0)
  const uint32_t following = row_rotated(choice, 1), third = row_rotated(choice, kMore);
  const bool near = l < top_k && !apart(choice, following);
  if (__any(near)) {
    const bool mixed = row_all(near ? 1 : 0, [](int a, int b) { return a | b; });
    const bool enough = l != top_k - 1 || apart(choice, third);
    sure = sure && (!mixed || row_all(enough ? 1 : 0, [](int a, int b) { return a & b; }));
    // the exact order of all but the last
    const bool there = l < top_k + kMore - 1 && choice != 0u;
    const float y = load_logit<XT>(logits, t * E + (there ? expert : 0));
    double exact = y;
    if (bias) {
      const double total = r.sigmoid ? 1.0 : softmax_sum(x, max);
      exact = is_masked(y) ? (double)y : score64(y, r.sigmoid, max, total) + (double)bias[there ? expert : 0];
    }
    const uint64_t mine = there ? order_key(exact) : 0ull;
    int rank = 0;
#pragma unroll
    for (int n = 1; n < kRow; ++n) {
      const uint64_t o = (uint64_t)row_rotated((unsigned long long)mine, n);
      const int e = row_rotated(expert, n);
      rank += o > mine || (o == mine && e < expert) ? 1 : 0;
    }
    const int sorted = __builtin_amdgcn_ds_permute(4 * (((int)threadIdx.x & 48) | (there ? rank : l)), expert);
    expert = mixed ? sorted : expert;
  }
  const bool used = l < top_k;
  const float chosen = used ? load_logit<XT>(logits, t * E + expert) : -inf;
  const double w = weight_of<kRow>(chosen, used, r.sigmoid, r.renormalize, max, sum);
  if (used && sure) {
    experts[t * top_k + l] = expert;
    weights[t * top_k + l] = (float)(w * (double)r.scale);
  }
  return sure;
}

// A workgroup kWaves x kRowTokens tokens; NJ 16 NJ >= E.
template <class XT, int NJ>
__global__ __launch_bounds__(kWaves * 64) void moe_route_kernel(const void* __restrict__ logits, int64_t T, Routing r,
                                                                const float* __restrict__ bias, int32_t* __restrict__ experts,
                                                                float* __restrict__ weights) {
  constexpr int kWide = (NJ + 3) / 4;
  __shared__ double keys[kWaves][64 * kWide], ranks[kWaves][64 * kWide];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * kRowTokens;
  if (t0 >= T) return;
  const int64_t t = t0 + (threadIdx.x >> 4 & 3);
  // rows past the last token work on it beside its own
  const bool sure = route_row<XT, NJ>(logits, t < T ? t : T - 1, r, bias, experts, weights);
  uint64_t left = __ballot(!sure);
  for (int i = 0; i < kRowTokens && t0 + i < T; ++i)
    if (left >> (16 * i) & 1) route_token<XT, kWide>(logits, t0 + i, r, bias, keys[wave], ranks[wave], experts, weights);
}

// The exact way alone, a wave a token; NJ: 64 NJ >= E.
template <class XT, int NJ>
__global__ __launch_bounds__(kWaves * 64) void moe_route_wide_kernel(const void* __restrict__ logits, int64_t T, Routing r,
                                                                     const float* __restrict__ bias,
                                                                     int32_t* __restrict__ experts, float* __restrict__ weights) {
  __shared__ double keys[kWaves][64 * NJ], ranks[kWaves][64 * NJ];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t < T) route_token<XT, NJ>(logits, t, r, bias, keys[wave], ranks[wave], experts, weights);
}

// dx[e] from dw: through w = scale s or scale s / (sum of the chosen s), and s.
//   softmax, renormalised: dx_c = scale p_c (dw_c - sum p dw), p = the weights over scale
//   softmax              : dx_e = s_e (scale dw_e - sum over the chosen of scale s dw)
//   sigmoid              : dx_c = scale dw_c s(x_c) s(-x_c), renormalised
//                          scale p_c (dw_c - sum p dw) s(-x_c)
// The differences dw_c - sum p dw (the p add up to 1) are taken with every dw as its distance
// from the largest logit's: where that one's p is nearly 1, its own difference is the sum of the
// others' small shares, and dw less a sum of nearly as much would leave nothing of it.
// Lane c works the chosen expert c out; then every expert adds up what names it.
// Bound by instructions, not by bytes: 8192 tokens of 64 experts, 6 of them, fp32 (4.8 MB, a
// microsecond) take 6.9 us (softmax; 230 vector instructions and 50 between lanes a token,
// which is a wave's), renormalised 6.7 (sigmoid 7.0).
template <class XT, int NJ>
__global__ __launch_bounds__(kWaves * 64) void moe_route_backward_kernel(const void* __restrict__ logits,
                                                                         const int32_t* __restrict__ experts,
                                                                         const float* __restrict__ dweights, int64_t T, int E,
                                                                         int top_k, int sigmoid, int renormalize, float scale,
                                                                         typename Int8Out<XT>::type* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t >= T) return;
  const int id = lane < top_k ? experts[t * top_k + lane] : -1;
  const bool used = id >= 0 && id < E;
  const float xc = used ? load_logit<XT>(logits, t * E + id) : -__builtin_inff();
  const double dw = used ? (double)dweights[t * top_k + lane] * (double)scale : 0.0;
  const bool all = !sigmoid && !renormalize;  // every logit has a part in the weights
  float x[NJ], max = -__builtin_inff();
  double s[NJ], sum = 0.0;
  if (all) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      x[j] = 64 * j + lane < E ? load_logit<XT>(logits, t * E + 64 * j + lane) : -__builtin_inff();
      max = fmaxf(max, x[j]);
    }
    max = team_max(max, 64);
    max = is_masked(max) ? 0.0f : max;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      s[j] = exp((double)x[j] - (double)max);
      sum += s[j];
    }
    sum = wave_sum(sum);
  }
  double d = dw;  // of the lane's chosen expert
  if (!all) {
    const float top = renormalize ? team_max(xc, 64) : 0.0f;
    const double p = weight_of(xc, used, sigmoid, renormalize, top, sum, true);
    if (renormalize) {
      const uint64_t at = __ballot(used && xc == top);
      const double from = dw - (at ? __shfl(dw, __builtin_ctzll(at), 64) : 0.0);
      d = from - wave_sum(used ? p * from : 0.0);
    }
    d *= sigmoid ? p * sigmoid64(-xc) : p;  // 1 - s would cancel next to 1
  }
  double dx[NJ] = {};
  for (int c = 0; c < top_k; ++c) {
    const int e = __shfl(id, c, 64);
    const double v = __shfl(d, c, 64);
#pragma unroll
    for (int j = 0; j < NJ; ++j) dx[j] += e == 64 * j + lane ? v : 0.0;
  }
  if (all) {
    double base = 0.0, dot = 0.0;
    bool found = false;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const uint64_t at = __ballot(x[j] == max);
      if (at && !found) base = __shfl(dx[j], __builtin_ctzll(at), 64), found = true;
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      dx[j] -= base;
      dot += s[j] * dx[j];
    }
    dot = sum == 0.0 ? 0.0 : wave_sum(dot) / sum;
#pragma unroll
    for (int j = 0; j < NJ; ++j) dx[j] = sum == 0.0 ? 0.0 : s[j] / sum * (dx[j] - dot);
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = 64 * j + lane;
    if (e < E) dlogits[t * E + e] = Int8Out<XT>::of((float)dx[j]);
  }
}

template <class F>
hipError_t by_experts(int E, F&& f) {
  if (E <= 64) return f(std::integral_constant<int, 1>{});
  if (E <= 128) return f(std::integral_constant<int, 2>{});
  return E <= 256 ? f(std::integral_constant<int, 4>{}) : f(std::integral_constant<int, 8>{});
}
template <class F>
hipError_t by_type(int dtype, F&& f) {
  return dtype == 0 ? f(F16{}) : (dtype == 1 ? f(BF16{}) : f(F32{}));
}

}  // namespace

int moe_route_max_experts() { return 512; }
int moe_route_max_top_k() { return 64; }

hipError_t launch_moe_route(const void* logits, int dtype, int64_t T, int E, int top_k, bool sigmoid, const float* bias,
                            int groups, int top_groups, int group_top, bool renormalize, float scale, int32_t* experts,
                            float* weights, hipStream_t stream) {
  const Routing r = {E, top_k, sigmoid, groups, top_groups, group_top, renormalize, scale};
  const int nj = (E + kRow - 1) / kRow;  // experts a lane of a row; groups are whole lanes
  const bool rows = top_k <= kRow - kMore && (groups == 1 || (kRow % groups == 0 && E % kRow == 0));
  return by_type(dtype, [&](auto tag) {
    using XT = decltype(tag);
    if (!rows)
      return by_experts(E, [&](auto n) {
        moe_route_wide_kernel<XT, decltype(n)::value><<<(unsigned)((T + kWaves - 1) / kWaves), kWaves * 64, 0, stream>>>(
            logits, T, r, bias, experts, weights);
        return hipGetLastError();
      });
    auto run = [&](auto n) {
      constexpr int kTokens = kWaves * kRowTokens;
      moe_route_kernel<XT, decltype(n)::value><<<(unsigned)((T + kTokens - 1) / kTokens), kWaves * 64, 0, stream>>>(
          logits, T, r, bias, experts, weights);
      return hipGetLastError();
    };
    return nj <= 4 ? run(std::integral_constant<int, 4>{}) : (nj <= 8 ? run(std::integral_constant<int, 8>{})
         : (nj <= 16 ? run(std::integral_constant<int, 16>{}) : run(std::integral_constant<int, 32>{})));
  });
}

hipError_t launch_moe_route_backward(const void* logits, int dtype, const int32_t* experts, const float* dweights, int64_t T,
                                     int E, int top_k, bool sigmoid, bool renormalize, float scale, void* dlogits,
                                     hipStream_t stream) {
  return by_type(dtype, [&](auto tag) {
    using XT = decltype(tag);
    return by_experts(E, [&](auto nj) {
      moe_route_backward_kernel<XT, decltype(nj)::value><<<(unsigned)((T + kWaves - 1) / kWaves), kWaves * 64, 0, stream>>>(
          logits, experts, dweights, T, E, top_k, sigmoid, renormalize, scale, static_cast<typename Int8Out<XT>::type*>(dlogits));
      return hipGetLastError();
    });
  });
}

}  // namespace woq
