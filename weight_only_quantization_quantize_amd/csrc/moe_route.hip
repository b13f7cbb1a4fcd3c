// Routing to experts, and its gradient.  Of a token's logits x[e]:
//   s = softmax(x) or sigmoid(x)
//   order of the experts: by x, or, with a bias b, by s + b in 64 bits; the lower index first
//     among equals; -infinity (a masked expert) after every number, a NaN last
//   groups: E / groups neighbours each; only the top_groups of them with the largest sum of
//     their group_top best keys (x or s + b; of two without a bias: s) are chosen from
//   w = scale s, over the sum of the chosen experts' s where that is asked for
//
// Bound by vector instructions: a logit is 2 or 4 bytes, its score and its part in the
// choice some fifty instructions a token's 256 experts.  So the usual routing (route_row) has
// four tokens a wave, 16 lanes each, NJ neighbouring experts a lane, and works in 32 bits:
//   scores p = 1 / (1 + 2^(-x log2 e)) and 2^((x - max) log2 e) / sum are off by at most 2^-20,
//   s + b by 2^-24 of itself more.  Two keys further apart than kClose (1 + |key|) = 2^-18
//   (1 + |key|) are in their right order, and so are two groups' sums further apart than
//   twice that.  Where a chosen key (or the best one left out), or the last group kept and
//   the best one dropped, are nearer than that (equal ones, infinities and NaN among them), the
//   token goes the exact way (route_token): a wave a token, keys in 64 bits.
// Without a bias the logits themselves are the keys, and exact.  More than 16 choices, or
// groups that are not whole lanes of experts, take the exact way at once.
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
// top_k); max, sum: of the row, as softmax without renormalisation needs them.
template <int TEAM = 64>
__device__ inline double weight_of(float x, bool used, bool sigmoid, bool renormalize, float max, double sum) {
  double s = 0.0;
  if (sigmoid) {
    if (used) s = sigmoid64(x);
  } else {
    if (renormalize) {  // the row's sum cancels
      max = used ? x : -__builtin_inff();
      max = team_max(max, TEAM);
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
constexpr float kClose = 0x1p-18f;

// A number's order as an unsigned one; the zeros are equal, a NaN comes below -infinity.
__device__ inline uint32_t order_key32(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 1u;
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ inline float key_value(uint32_t k) {
  return __builtin_bit_cast(float, k <= 1u ? 0x7FC00000u : ((k >> 31) ? k & 0x7FFFFFFFu : ~k));
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
template <class T>
__device__ inline T row_rotated(T v, int n) {  // of the lane n further on
  return __shfl(v, ((int)threadIdx.x & 48) | (((int)threadIdx.x + n) & 15), 64);
}

// Four tokens by a wave, lane l of a row of 16 the n = ceil(E / 16) experts from l n on, n <=
// NJ.  Returns whether the row's choice is exact; then it is written.
template <class XT, int NJ>
__device__ __forceinline__ bool route_row(const void* __restrict__ logits, int64_t t, const Routing& r,
                                          const float* __restrict__ bias, int32_t* __restrict__ experts,
                                          float* __restrict__ weights) {
  constexpr float kLog2e = 1.44269504088896341f;
  const int E = r.E, top_k = r.top_k, l = threadIdx.x & (kRow - 1), n = (E + kRow - 1) / kRow, e0 = l * n;
  const int own = E - e0 < n ? E - e0 : n;  // of the lane; the rest counts as masked
  const float inf = __builtin_inff();
  float x[NJ], max = -inf;
  constexpr int kVector = kElementBytes<XT> == 4 || NJ < 8 ? 4 : 8;  // elements a load, of any alignment
#pragma unroll
  for (int j0 = 0; j0 < NJ; j0 += kVector) {
    if (j0 + kVector <= own) {
      typename Int8Out<XT>::type v[kVector];
      __builtin_memcpy(v, static_cast<const typename Int8Out<XT>::type*>(logits) + t * E + e0 + j0, sizeof(v));
#pragma unroll
      for (int j = 0; j < kVector; ++j) x[j0 + j] = load_logit<XT>(v, j);
    } else {
#pragma unroll
      for (int j = j0; j < j0 + kVector; ++j) x[j] = j < own ? load_logit<XT>(logits, t * E + e0 + j) : -inf;
    }
  }
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
  if (all) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) sum += exp((double)x[j] - (double)max);
    sum = wave_sum<kRow>(sum);
  }
  float by[NJ];  // what groups are compared by
  uint32_t key[NJ];
  if (scored) {
    float part = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      by[j] = __builtin_amdgcn_exp2f((r.sigmoid ? -x[j] : x[j] - max) * kLog2e);
      part += by[j];
    }
    float inverse = 0.0f;
    if (!r.sigmoid) inverse = __builtin_amdgcn_rcpf(row_all(part, [](float a, float b) { return a + b; }));
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      by[j] = r.sigmoid ? __builtin_amdgcn_rcpf(1.0f + by[j]) : by[j] * inverse;
      if (bias) by[j] += bias[j < own ? e0 + j : 0];
      by[j] = is_masked(x[j]) ? x[j] : by[j];
      key[j] = j < own ? order_key32(bias ? by[j] : x[j]) : 0u;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      by[j] = x[j];
      key[j] = j < own ? order_key32(x[j]) : 0u;
    }
  }
  bool sure = true;
  if (r.groups > 1) {  // a group is kRow / groups lanes
    float best = -inf, next = -inf;
    bool odd = false;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      odd |= by[j] != by[j];
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
    int before = 0;
#pragma unroll
    for (int n = 1; n < kRow; ++n) before += row_rotated(rank, n) > rank ? 1 : 0;
    const bool kept = before < r.top_groups * lanes;
    if (!kept)
#pragma unroll
      for (int j = 0; j < NJ; ++j) key[j] = 0u;
    const float last = -row_all(kept ? -rank : -inf, larger), first = row_all(kept ? -inf : rank, larger);
    // (one group's best alone is exact where it is a logit; equal ones are not told apart here)
    const float close = bias || r.group_top > 1 ? 2.0f * kClose * (1.0f + fabsf(last)) : 0.0f;
    const int keeps = row_all(kept ? 1 : 0, [](int a, int b) { return a + b; });
    sure = r.top_groups == r.groups || (last - first > close && keeps == r.top_groups * lanes);
    sure = sure && !row_all(odd ? 1 : 0, [](int a, int b) { return a | b; });
  }
  int expert = 0;
  float before = inf;
  const int rounds = bias ? top_k + 1 : top_k;  // with the best one left out
  for (int c = 0; c < rounds; ++c) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) m = key[j] > m ? key[j] : m;
    m = row_all(m, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    if (bias) {
      const float v = key_value(m);
      if (c > 0 && m > 0u) sure = sure && before - v > kClose * (1.0f + fabsf(v));
      before = v;
    }
    int id = 1 << 20;  // the lowest index of that key
#pragma unroll
    for (int j = NJ - 1; j >= 0; --j) id = key[j] == m && j < own ? e0 + j : id;
    id = row_all(id, [](int a, int b) { return a < b ? a : b; });
    const int mine = id - e0;  // outside 0 .. n - 1: another lane's
#pragma unroll
    for (int j = 0; j < NJ; ++j) key[j] = mine == j ? 0u : key[j];
    expert = l == c ? id : expert;
  }
  const bool used = l < top_k;
  const float chosen = used && expert < E ? load_logit<XT>(logits, t * E + expert) : -inf;
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
//   sigmoid              : dx_c = ds_c s_c (1 - s_c), ds_c = scale dw_c, renormalised
//                          scale (dw_c - sum p dw) / (sum of s)
// Lane c works the chosen expert c out; then every expert adds up what names it.
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
  const double p = weight_of(xc, used, sigmoid, renormalize, max, sum);
  const double dot = wave_sum(used ? p * dw : 0.0);
  double d;  // of the lane's chosen expert
  if (all) {
    d = dw;
  } else if (!sigmoid) {
    d = p * (dw - dot);
  } else {
    const double score = used ? sigmoid64(xc) : 0.0;
    if (renormalize) {
      const double total = wave_sum(score);
      d = total == 0.0 ? 0.0 : (dw - dot) / total * score * (1.0 - score);
    } else {
      d = dw * score * (1.0 - score);
    }
  }
  double dx[NJ] = {};
  for (int c = 0; c < top_k; ++c) {
    const int e = __shfl(id, c, 64);
    const double v = __shfl(d, c, 64);
#pragma unroll
    for (int j = 0; j < NJ; ++j) dx[j] += e == 64 * j + lane ? v : 0.0;
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = 64 * j + lane;
    if (all) dx[j] = sum == 0.0 ? 0.0 : s[j] / sum * (dx[j] - dot);
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
  const bool rows = top_k <= kRow && (groups == 1 || (kRow % groups == 0 && E % kRow == 0));
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
