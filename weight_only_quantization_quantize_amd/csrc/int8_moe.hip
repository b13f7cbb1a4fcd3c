// A layer of gated experts with 8-bit integer weights, for tokens that are routed already:
//   q, a   = the codes and scales of X's rows (int8_quantize)
//   g, u   = (acc a[t]) s_up[e, .] of the gate and the up rows of up[e], acc = sum_k q[t, k] up[e, ., k]
//   h      = silu(g) u, silu(g) = g / (1 + exp(-g)), fp32; quantised by rows again: p, b
//   y[t,c] = (acc b) s_down[e, .],  acc = sum_i p[i] down[e, ., i]
//   Y[t]   = sum over the token's choices c of weights[t, c] y[t, c], rounded once
// A choice whose expert is none of 0 .. E - 1 is left out.
//
// Launches: the rows of X are quantised; `plan` sorts the choices by expert into rows and
// cuts each expert's rows into tiles; `up` and `down` are tile products (int8_tile.h) over
// those tiles; h's rows are quantised between them; `combine` adds up.  The rows' order in
// the plan changes no result: every row is computed by itself.
#include "int8_tile.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kMaxExperts = 512;
constexpr int kPlanThreads = 1024;

// Up to BM rows of an expert.
struct Tile {
  int expert, row, count;
};
struct Plan {
  int tiles;
};

// One workgroup.  where [T top_k]: a choice's row, -1 of none; token [rows].
__global__ __launch_bounds__(kPlanThreads) void int8_moe_plan_kernel(const int32_t* __restrict__ experts, int choices,
                                                                    int top_k, int E, int BM, Plan* __restrict__ plan,
                                                                    Tile* __restrict__ tiles, int* __restrict__ where,
                                                                    int* __restrict__ token) {
  __shared__ int count[kMaxExperts], first[kMaxExperts], tile[kMaxExperts];
  for (int e = threadIdx.x; e < E; e += kPlanThreads) count[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < choices; i += kPlanThreads) {
    const int e = experts[i];
    if (e >= 0 && e < E) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int rows = 0, of = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane, n = e < E ? count[e] : 0, m = (n + BM - 1) / BM;
      int upto = n, tupto = m;
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(upto, off, 64), p = __shfl_up(tupto, off, 64);
        if (lane >= off) upto += o, tupto += p;
      }
      if (e < E) first[e] = rows + upto - n, tile[e] = of + tupto - m;
      rows += __shfl(upto, 63, 64);
      of += __shfl(tupto, 63, 64);
    }
    if (lane == 0) plan->tiles = of;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kPlanThreads) {
    for (int i = 0; i * BM < count[e]; ++i) {
      const int left = count[e] - i * BM;
      tiles[tile[e] + i] = Tile{e, first[e] + i * BM, left < BM ? left : BM};
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < choices; i += kPlanThreads) {
    const int e = experts[i];
    int row = -1;
    if (e >= 0 && e < E) {
      row = atomicAdd(&first[e], 1);
      token[row] = i / top_k;
    }
    where[i] = row;
  }
}

// UP: A = X's codes, gathered; W's tile is blocks of 32 gate rows and the 32 up rows of the
// same columns in turn.  Else A = h's codes.  ntiles: of columns of h (of y).
template <bool UP, class C>
__global__ __launch_bounds__(C::kThreads, C::kOccupancy) void int8_moe_product_kernel(
    const int8_t* __restrict__ A, const float* __restrict__ sa, const int8_t* __restrict__ W, const float* __restrict__ sw,
    const Plan* __restrict__ plan, const Tile* __restrict__ tiles, const int* __restrict__ token, int K, int N, int ntiles,
    float* __restrict__ out) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kLdsBytes];
  const int mt = (int)blockIdx.x / ntiles, n0 = (int)blockIdx.x % ntiles * (UP ? C::BN / 2 : C::BN);
  if (mt >= plan->tiles) return;
  const Tile tile = tiles[mt];
  const int rows = UP ? 2 * N : N;  // of an expert's weights
  const int8_t* const w = W + (int64_t)tile.expert * rows * K;
  const float* const s = sw + (int64_t)tile.expert * rows;
  auto clamped = [&](int r) { return r < tile.count ? r : tile.count - 1; };
  typename C::Sums acc;
  const bool mine = C::multiply(
      acc, lds, UP ? A : A + (int64_t)tile.row * K,
      [&](int r) { return (uint32_t)(UP ? token[tile.row + clamped(r)] : clamped(r)) * (uint32_t)K; }, w,
      [&](int r) {
        const int n = UP ? n0 + (r >> 6) * 32 + (r & 31) : n0 + r;
        return ((uint32_t)(n < N ? n : N - 1) + (UP && (r & 32) ? (uint32_t)N : 0u)) * (uint32_t)K;
      },
      K);
  if (!mine) return;

  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kCols = UP ? 16 * C::TN : 32 * C::TN;
  constexpr int kTurn = 32 * (kCols * 4 + 16) + kCols * 8;
  static_assert(C::kWaves * kTurn <= C::kStages * C::kStage, "the turn fits the stages' place");
  static_assert(!UP || C::TN % 2 == 0, "a wave has gate and up columns");
  const int m1 = wave % C::WM * (32 * C::TM), n1 = n0 + wave / C::WM * kCols;
  uint8_t* const turn = lds + wave * kTurn;
  float* const cols = reinterpret_cast<float*>(turn + 32 * (kCols * 4 + 16));
  for (int c = lane; c < kCols; c += 64) {
    const int n = n1 + c < N ? n1 + c : N - 1;
    cols[c] = s[n];
    if (UP) cols[kCols + c] = s[N + n];
  }
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < C::TM; ++i) {
    const int m = m1 + 32 * i, r = clamped(m + (lane & 31));
    if (m >= tile.count) break;
    const float f = sa[UP ? token[tile.row + r] : tile.row + r];
    int8_store_rows<F32, kCols>(turn, out + (int64_t)(tile.row + m) * N + n1, N, tile.count - m, N - n1, [&](int b) {
      const float4_t c = *reinterpret_cast<const float4_t*>(cols + 8 * b + 4 * half);
      float4_t v;
      if constexpr (UP) {
        const float4_t d = *reinterpret_cast<const float4_t*>(cols + kCols + 8 * b + 4 * half);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float g = (float)acc[i][b / 4 * 2][4 * (b % 4) + e] * f * c[e];
          const float u = (float)acc[i][b / 4 * 2 + 1][4 * (b % 4) + e] * f * d[e];
          v[e] = g / (1.0f + expf(-g)) * u;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][b / 4][4 * (b % 4) + e] * f * c[e];
      }
      return v;
    });
  }
}

// Y[t] = the sum of its choices' rows of `products`, weighted, in the order of choice.
template <class YT>
__global__ __launch_bounds__(256) void int8_moe_combine_kernel(const float* __restrict__ products, const int* __restrict__ where,
                                                               const float* __restrict__ weights, int T, int H, int top_k,
                                                               uint16_t* __restrict__ Y) {
  const int n = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 4;
  if (n >= H) return;
  for (int t = (int)blockIdx.y; t < T; t += (int)gridDim.y) {
    float4_t v = {};
    for (int c = 0; c < top_k; ++c) {
      const int row = where[(int64_t)t * top_k + c];
      if (row < 0) continue;
      const float w = weights[(int64_t)t * top_k + c];
      const float4_t p = *reinterpret_cast<const float4_t*>(products + (int64_t)row * H + n);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += w * p[e];
    }
    const uint32_t lo = (uint32_t)YT::from_f32(v[0]) | (uint32_t)YT::from_f32(v[1]) << 16;
    const uint32_t hi = (uint32_t)YT::from_f32(v[2]) | (uint32_t)YT::from_f32(v[3]) << 16;
    *reinterpret_cast<u32x2_t*>(Y + (int64_t)t * H + n) = u32x2_t{lo, hi};
  }
}

typedef Int8Tile<1, 2, 2, 4, 1, 3> Small;
typedef Int8Tile<2, 2, 2, 4, 1, 2> Middle;

// Tiles of rows, at most: one for each expert that is taken and one for each further BM.
int64_t most_tiles(int64_t choices, int64_t E, int64_t BM) { return (choices < E ? choices : E) + choices / BM; }
int64_t tile_rows(int64_t T, int64_t E, int64_t top_k) { return T * top_k <= 64 * E ? Small::BM : Middle::BM; }

struct Layout {
  size_t codes, scales, plan, tiles, where, token, h, h_codes, h_scales, products, bytes;
};
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
Layout layout(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k) {
  const size_t rows = (size_t)(T * top_k);
  Layout l;
  l.codes = 0;
  l.scales = up256((size_t)(T * H));
  l.plan = up256(l.scales + (size_t)T * 4);
  l.tiles = l.plan + 256;
  l.where = up256(l.tiles + (size_t)most_tiles(T * top_k, E, tile_rows(T, E, top_k)) * sizeof(Tile));
  l.token = up256(l.where + rows * 4);
  l.h = up256(l.token + rows * 4);
  l.h_codes = up256(l.h + rows * (size_t)I * 4);
  l.h_scales = up256(l.h_codes + rows * (size_t)I);
  l.products = up256(l.h_scales + rows * 4);
  l.bytes = l.products + rows * (size_t)H * 4;
  return l;
}

}  // namespace

int int8_moe_max_experts() { return kMaxExperts; }

size_t int8_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k) {
  return layout(T, H, I, E, top_k).bytes;
}

hipError_t launch_int8_moe(const void* X, int xdtype, const int32_t* experts, const float* weights, const void* up,
                           const float* up_scales, const void* down, const float* down_scales, int64_t T, int64_t H, int64_t I,
                           int64_t E, int top_k, void* Y, void* workspace, hipStream_t stream) {
  const Layout l = layout(T, H, I, E, top_k);
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  const int64_t choices = T * top_k, BM = tile_rows(T, E, top_k);
  Plan* const plan = reinterpret_cast<Plan*>(ws + l.plan);
  Tile* const tiles = reinterpret_cast<Tile*>(ws + l.tiles);
  int* const where = reinterpret_cast<int*>(ws + l.where);
  int* const token = reinterpret_cast<int*>(ws + l.token);
  float* const h = reinterpret_cast<float*>(ws + l.h);
  float* const products = reinterpret_cast<float*>(ws + l.products);
  float* const h_scales = reinterpret_cast<float*>(ws + l.h_scales);
  float* const x_scales = reinterpret_cast<float*>(ws + l.scales);
  hipError_t e = launch_int8_quantize(X, xdtype, nullptr, false, T, H, ws + l.codes, x_scales, stream);
  if (e != hipSuccess) return e;
  int8_moe_plan_kernel<<<1, kPlanThreads, 0, stream>>>(experts, (int)choices, top_k, (int)E, (int)BM, plan, tiles, where, token);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t mt = most_tiles(choices, E, BM);
  auto product = [&](auto is_up, auto tag, const void* a, const float* sa, const void* w, const float* sw, int64_t K, int64_t N,
                     float* out) {
    using C = decltype(tag);
    constexpr bool kUp = decltype(is_up)::value;
    constexpr int kCols = kUp ? C::BN / 2 : C::BN;
    const int64_t nt = (N + kCols - 1) / kCols;
    int8_moe_product_kernel<kUp, C><<<(unsigned)(mt * nt), C::kThreads, 0, stream>>>(
        static_cast<const int8_t*>(a), sa, static_cast<const int8_t*>(w), sw, plan, tiles, token, (int)K, (int)N, (int)nt, out);
    return hipGetLastError();
  };
  auto products_of = [&](auto tag) {
    hipError_t e = product(std::true_type{}, tag, ws + l.codes, x_scales, up, up_scales, H, I, h);
    if (e != hipSuccess) return e;
    e = launch_int8_quantize(h, 2, nullptr, false, choices, I, ws + l.h_codes, h_scales, stream);
    if (e != hipSuccess) return e;
    return product(std::false_type{}, tag, ws + l.h_codes, h_scales, down, down_scales, I, H, products);
  };
  e = BM == Small::BM ? products_of(Small{}) : products_of(Middle{});
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((H + 1023) / 1024), (unsigned)(T < 65535 ? T : 65535));
  auto* const f = xdtype == 0 ? int8_moe_combine_kernel<F16> : int8_moe_combine_kernel<BF16>;
  f<<<grid, 256, 0, stream>>>(products, where, weights, (int)T, (int)H, top_k, static_cast<uint16_t*>(Y));
  return hipGetLastError();
}

}  // namespace woq
