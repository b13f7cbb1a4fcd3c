// Products of two 8-bit integer matrices with a scale for each row of either:
//   Y[m, n] = (acc sa[m]) sw[n] + bias[n],  acc = sum_k a[m, k] w[n, k]
// The sums are exact (int8_tile.h); the scales multiply in fp32, Y is rounded once.
#include "int8_tile.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kXcds = 8;
constexpr int kGroup = 8;  // M tiles of a group

// Tile order.  Workgroup b runs on XCD b % 8; each XCD takes one contiguous run of tiles,
// in groups of 8 M tiles, M fastest, so that the tiles in flight there share about as much
// of A as of W in its L2.
template <class YT, class C>
__global__ __launch_bounds__(C::kThreads, 2) void int8_gemm_kernel(
    const int8_t* __restrict__ A, const float* __restrict__ sa, const int8_t* __restrict__ W, const float* __restrict__ sw,
    const float* __restrict__ bias, int M, int N, int K, int mtiles, int tiles, typename Int8Out<YT>::type* __restrict__ Y) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kLdsBytes];
  const int per = (tiles + kXcds - 1) / kXcds;
  const int tile = (int)(blockIdx.x % kXcds) * per + (int)(blockIdx.x / kXcds);
  if (tile >= tiles) return;
  const int gtiles = kGroup * (tiles / mtiles);  // of a group of M tiles
  const int g = tile / gtiles, gm = mtiles - g * kGroup < kGroup ? mtiles - g * kGroup : kGroup;
  const int m0 = (g * kGroup + tile % gtiles % gm) * C::BM, n0 = tile % gtiles / gm * C::BN;
  typename C::Sums acc;
  const bool mine = C::multiply(
      acc, lds, A + (int64_t)m0 * K, [&](int r) { return (uint32_t)((m0 + r < M ? r : M - 1 - m0) * K); },
      W + (int64_t)n0 * K, [&](int r) { return (uint32_t)((n0 + r < N ? r : N - 1 - n0) * K); }, K);
  if (!mine) return;

  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m1 = m0 + (wave & 1) * (32 * C::TM), n1 = n0 + (wave >> 1) * (32 * C::TN);
  constexpr int kCols = 32 * C::TN, kTurn = 32 * (kCols * 4 + 16) + kCols * 8;
  // a wave's LDS: the turn, then its columns' scales and biases
  static_assert(C::kWaves * kTurn <= C::kStages * C::kStage, "the turn fits the stages' place");
  uint8_t* const turn = lds + wave * kTurn;
  float* const cols = reinterpret_cast<float*>(turn + 32 * (kCols * 4 + 16));
  for (int c = lane; c < kCols; c += 64) {
    const int n = n1 + c < N ? n1 + c : N - 1;
    cols[c] = sw[n];
    cols[kCols + c] = bias ? bias[n] : 0.0f;
  }
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < C::TM; ++i) {
    const int m = m1 + 32 * i, r = m + (lane & 31);
    if (m >= M) break;
    const float f = sa[r < M ? r : M - 1];
    int8_store_rows<YT, kCols>(turn, Y + (int64_t)m * N + n1, N, M - m, N - n1, [&](int b) {
      const float4_t s = *reinterpret_cast<const float4_t*>(cols + 8 * b + 4 * half);
      const float4_t t = *reinterpret_cast<const float4_t*>(cols + kCols + 8 * b + 4 * half);
      float4_t v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][b / 4][4 * (b % 4) + e] * f * s[e] + t[e];
      return v;
    });
  }
}

template <class YT, class C>
hipError_t launch_tiles(const int8_t* A, const float* sa, const int8_t* W, const float* sw, const float* bias, int64_t M,
                        int64_t N, int64_t K, void* Y, hipStream_t stream) {
  const int64_t mt = (M + C::BM - 1) / C::BM, nt = (N + C::BN - 1) / C::BN, tiles = mt * nt;
  const unsigned grid = (unsigned)((tiles + kXcds - 1) / kXcds * kXcds);
  int8_gemm_kernel<YT, C><<<grid, C::kThreads, 0, stream>>>(A, sa, W, sw, bias, (int)M, (int)N, (int)K, (int)mt, (int)tiles,
                                                           static_cast<typename Int8Out<YT>::type*>(Y));
  return hipGetLastError();
}

int64_t per_cu(int64_t M, int64_t N, int bm, int bn) { return ((M + bm - 1) / bm * ((N + bn - 1) / bn) + 255) / 256; }

template <class YT>
hipError_t launch(const int8_t* A, const float* sa, const int8_t* W, const float* sw, const float* bias, int64_t M,
                  int64_t N, int64_t K, void* Y, hipStream_t stream) {
  const double large = 48.0 * per_cu(M, N, 256, 256), mid = 6.0 + 14.0 * per_cu(M, N, 128, 128),
               small = 3.0 + 6.0 * per_cu(M, N, 64, 64);
  if (large <= mid && large <= small) return launch_tiles<YT, Int8Tile<4, 2, 4, 4, 1>>(A, sa, W, sw, bias, M, N, K, Y, stream);
  if (mid <= small) return launch_tiles<YT, Int8Tile<2, 2, 2, 4, 1>>(A, sa, W, sw, bias, M, N, K, Y, stream);
  return launch_tiles<YT, Int8Tile<1, 1, 2, 4, 2>>(A, sa, W, sw, bias, M, N, K, Y, stream);
}

}  // namespace

hipError_t launch_int8_gemm(const void* A, const float* a_scales, const void* W, const float* w_scales, const float* bias,
                            int64_t M, int64_t N, int64_t K, int ydtype, void* Y, hipStream_t stream) {
  auto* const f = ydtype == 0 ? launch<F16> : (ydtype == 1 ? launch<BF16> : launch<F32>);
  return f(static_cast<const int8_t*>(A), a_scales, static_cast<const int8_t*>(W), w_scales, bias, M, N, K, Y, stream);
}

namespace {
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
}  // namespace

size_t int8_linear_workspace_bytes(int64_t M, int64_t, int64_t K) { return up256((size_t)(M * K)) + (size_t)M * 4; }

hipError_t launch_int8_linear(const void* X, int xdtype, const float* act_scale, const void* W, const float* w_scales,
                              const float* bias, int64_t M, int64_t N, int64_t K, void* Y, void* workspace, hipStream_t stream) {
  float* const scales = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + up256((size_t)(M * K)));
  const hipError_t e = launch_int8_quantize(X, xdtype, act_scale, false, M, K, workspace, scales, stream);
  if (e != hipSuccess) return e;
  return launch_int8_gemm(workspace, scales, W, w_scales, bias, M, N, K, xdtype, Y, stream);
}

}  // namespace woq
