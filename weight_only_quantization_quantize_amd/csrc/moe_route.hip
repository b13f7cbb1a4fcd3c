// Routing to experts, and its gradient.  Of a token's logits x[e]:
//   s = softmax(x) or sigmoid(x)
//   order of the experts: by x, or, with a bias b, by s + b in 64 bits; the lower index first
//     among equals; -infinity (a masked expert) after every number, a NaN last
//   groups: E / groups neighbours each; only the top_groups of them with the largest sum of
//     their group_top best keys (x or s + b; of two without a bias: s) are chosen from
//   w = scale s, over the sum of the chosen experts' s where that is asked for
// A wave a token; lane l holds the experts 64 j + l.
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
__device__ inline double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
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

// The weights of the chosen experts' logits, lane c holding the c-th (used: c < top_k);
// max, sum: of the row, as softmax without renormalisation needs them.
__device__ inline double weight_of(float x, bool used, bool sigmoid, bool renormalize, float max, double sum) {
  double s = 0.0;
  if (sigmoid) {
    if (used) s = sigmoid64(x);
  } else {
    if (renormalize) {  // the row's sum cancels
      max = used ? x : -__builtin_inff();
      max = team_max(max, 64);
      max = is_masked(max) ? 0.0f : max;
    }
    if (used) s = exp((double)x - (double)max);
  }
  if (renormalize) sum = wave_sum(s);
  if (sigmoid && !renormalize) return s;
  return sum == 0.0 ? 0.0 : s / sum;
}

// NJ: 64 NJ >= E.
template <class XT, int NJ>
__global__ __launch_bounds__(kWaves * 64) void moe_route_kernel(const void* __restrict__ logits, int64_t T, int E, int top_k,
                                                                int sigmoid, const float* __restrict__ bias, int groups,
                                                                int top_groups, int group_top, int renormalize, float scale,
                                                                int32_t* __restrict__ experts, float* __restrict__ weights) {
  __shared__ double keys_all[kWaves][64 * NJ];
  __shared__ double ranks_all[kWaves][64 * NJ];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t >= T) return;
  float x[NJ], max = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    x[j] = 64 * j + lane < E ? load_logit<XT>(logits, t * E + 64 * j + lane) : -__builtin_inff();
    max = fmaxf(max, x[j]);
  }
  max = team_max(max, 64);
  max = is_masked(max) ? 0.0f : max;
  double s[NJ], sum = 0.0;
  const bool wide = bias || (groups > 1 && group_top > 1);  // scores of all experts
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
    double k = x[j], r = x[j];
    if (wide) {
      const double p = sigmoid || sum == 0.0 ? s[j] : s[j] / sum;
      if (bias)
        r = k = is_masked(x[j]) ? (double)x[j] : p + (double)bias[e < E ? e : 0];
      else
        r = is_masked(x[j]) ? (double)x[j] : p;
    }
    key[j] = e < E ? order_key(k) : 0ull;
    if (groups > 1) keys_all[wave][e] = r;
  }
  if (groups > 1) {
    // lane g: groups g, g + 64, ...
    const double* const keys = keys_all[wave];
    double* const ranks = ranks_all[wave];
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
      ranks[g] = group_top > 1 ? best + next : best;
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
      if (before >= top_groups) key[j] = 0ull;
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
    weights[t * top_k + lane] = (float)(w * (double)scale);
  }
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
  return by_type(dtype, [&](auto tag) {
    return by_experts(E, [&](auto nj) {
      moe_route_kernel<decltype(tag), decltype(nj)::value><<<(unsigned)((T + kWaves - 1) / kWaves), kWaves * 64, 0, stream>>>(
          logits, T, E, top_k, sigmoid, bias, groups, top_groups, group_top, renormalize, scale, experts, weights);
      return hipGetLastError();
    });
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
