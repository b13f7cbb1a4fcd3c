// Products of two 8-bit integer matrices with a scale for each row of either:
//   Y[m, n] = (acc sa[m]) sw[n] + bias[n],  acc = sum_k a[m, k] w[n, k]
// The sums are exact (int8_tile.h, which says what bounds them); the first scale multiplies in
// fp32, the second one and the bias (0 where there is none) in one fma, here and in
// int8_gemv.hip, so that an element has the same bits whichever kernel takes it; Y is rounded
// once.  Few rows go to the kernel that streams the weights past them (int8_gemv.hip): up to
// four with K <= 8192, one with K <= 32768.
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
__global__ __launch_bounds__(C::kThreads, C::kOccupancy) void int8_gemm_kernel(
    const int8_t* __restrict__ A, const float* __restrict__ sa, const int8_t* __restrict__ W, const float* __restrict__ sw,
    const float* __restrict__ bias, int M, int N, int K, int mtiles, int tiles, typename Int8Out<YT>::type* __restrict__ Y) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kLdsBytes];
  const int per = (tiles + kXcds - 1) / kXcds;
  const int tile = (int)(blockIdx.x % kXcds) * per + (int)(blockIdx.x / kXcds);
  if (tile >= tiles) return;
  const int gtiles = kGroup * (tiles / mtiles);  // of a group of M tiles
  const int g = tile / gtiles, gm = mtiles - g * kGroup < kGroup ? mtiles - g * kGroup : kGroup;
  const int m0 = (g * kGroup + tile % gtiles % gm) * C::BM, n0 = tile % gtiles / gm * C::BN;
  C::for_blocks(M - m0, [&](auto blocks) {
    constexpr int kBlocks = decltype(blocks)::value;
    typename C::template Sums<kBlocks> acc;
    const bool mine = C::template multiply<kBlocks>(
        acc, lds, A + (int64_t)m0 * K, [&](int r) { return (uint32_t)((m0 + r < M ? r : M - 1 - m0) * K); },
        W + (int64_t)n0 * K, [&](int r) { return (uint32_t)((n0 + r < N ? r : N - 1 - n0) * K); }, K);
    if (!mine) return;

    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n1 = n0 + wave / C::WM * (32 * C::TN);
    constexpr int kCols = 32 * C::TN, kPitch = kCols * (int)sizeof(*Y) + 16, kTurn = 32 * kPitch + kCols * 8;
    // a wave's LDS: the turn, then its columns' scales and biases
    static_assert(C::kWaves * kTurn <= C::kGroupBytes, "the turn fits the stages' place");
    uint8_t* const turn = lds + wave * kTurn;
    float* const cols = reinterpret_cast<float*>(turn + 32 * kPitch);
    for (int c = lane; c < kCols; c += 64) {
      const int n = n1 + c < N ? n1 + c : N - 1;
      cols[c] = sw[n];
      cols[kCols + c] = bias ? bias[n] : 0.0f;
    }
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const int m = m0 + 32 * C::row_block(wave, i), r = m + (lane & 31);
      if (m >= M) break;
      const float f = sa[r < M ? r : M - 1];
      int8_store_rows<YT, kCols>(turn, Y + (int64_t)m * N + n1, N, M - m, N - n1, [&](int b) {
        const float4_t s = *reinterpret_cast<const float4_t*>(cols + 8 * b + 4 * half);
        const float4_t t = *reinterpret_cast<const float4_t*>(cols + kCols + 8 * b + 4 * half);
        float4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fmaf((float)acc[i][b / 4][4 * (b % 4) + e] * f, s[e], t[e]);
        return v;
      });
    }
  });
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

// The tile with the smallest time by a model of what was measured (weights out of HBM, 327
// sizes from 2 x 36 x 64 to 4096 x 11008 x 4096, and 260 small ones), in us for r tiles a
// compute unit and s stages of 128 K:  fixed + r (tile + stage s).  The choice takes 3% more
// than the fastest of all in the mean, of the small ones 0.5%.  Large tiles read LDS least for
// a matrix instruction (2048 x 11008 x 4096: 256 x 384 85 us, 192 x 256 95, 128 x 128 107,
// 256 x 256, whose 344 tiles fill two rounds badly, 111; 8192 x 8192 x 8192: 459, 510, 539 and
// 450); small ones are there for outputs of few tiles, where K is split between four groups
// of waves and many stages are in flight (16 x 4096 x 11008: 32 x 32 16.4 us, 64 x 32 18.1, 64 x 64 23.7; 128 x 4096 x 4096:
// 15, 9.3 and 10.4; 16 x 28672 x 8192: 55, 58 and 45.5).
struct Model {
  int bm, bn;
  double fixed, tile, stage;
};
constexpr Model kModels[] = {{256, 256, 0.0, 7.95, 1.24}, {256, 384, 0.0, 11.08, 1.73}, {192, 256, 0.0, 6.61, 1.02},
                             {128, 256, 0.0, 5.91, 0.75}, {128, 128, 0.0, 5.17, 0.47},  {64, 128, 0.19, 3.24, 0.35},
                             {64, 64, 1.9, 1.3, 0.24},    {32, 64, 2.44, 1.08, 0.22},   {64, 32, 0.85, 3.46, 0.18},
                             {32, 32, 1.19, 2.84, 0.15}};
int choose(int64_t M, int64_t N, int64_t K) {
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < (int)(sizeof(kModels) / sizeof(kModels[0])); ++i) {
    const Model& m = kModels[i];
    const double r = (double)(((M + m.bm - 1) / m.bm * ((N + m.bn - 1) / m.bn) + 255) / 256);
    const double t = m.fixed + r * (m.tile + m.stage * (double)((K + 127) / 128));
    if (i == 0 || t < least) least = t, best = i;
  }
  return best;
}

template <class YT>
hipError_t launch(const int8_t* A, const float* sa, const int8_t* W, const float* sw, const float* bias, int64_t M,
                  int64_t N, int64_t K, void* Y, hipStream_t stream) {
  auto run = [&](auto tag) { return launch_tiles<YT, decltype(tag)>(A, sa, W, sw, bias, M, N, K, Y, stream); };
  switch (choose(M, N, K)) {
    case 0: return run(Int8Tile<4, 2, 4, 4, 1, 2>{});
    case 1: return run(Int8Tile<4, 3, 4, 4, 1, 2>{});
    case 2: return run(Int8Tile<3, 2, 4, 4, 1, 2>{});
    case 3: return run(Int8Tile<2, 2, 4, 4, 1, 3>{});
    case 4: return run(Int8Tile<2, 2, 2, 4, 1, 4, 1>{});
    case 5: return run(Int8Tile<1, 1, 4, 4, 1, 4>{});
    case 6: return run(Int8Tile<1, 1, 2, 4, 1, 4>{});
    case 7: return run(Int8Tile<1, 1, 2, 4, 1, 6, 1, 1>{});
    case 8: return run(Int8Tile<1, 1, 1, 4, 4, 3>{});
    default: return run(Int8Tile<1, 1, 1, 4, 4, 4, 1, 1>{});
  }
}

}  // namespace

hipError_t launch_int8_gemm(const void* A, const float* a_scales, const void* W, const float* w_scales, const float* bias,
                            int64_t M, int64_t N, int64_t K, int ydtype, void* Y, hipStream_t stream) {
  if (M <= int8_gemv_max_rows(K)) return launch_int8_gemv(A, a_scales, W, w_scales, bias, M, N, K, ydtype, Y, stream);
  auto* const f = ydtype == 0 ? launch<F16> : (ydtype == 1 ? launch<BF16> : launch<F32>);
  return f(static_cast<const int8_t*>(A), a_scales, static_cast<const int8_t*>(W), w_scales, bias, M, N, K, Y, stream);
}

namespace {
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
}  // namespace

// The rows' codes and scales, or nothing where one launch does it all.
size_t int8_linear_workspace_bytes(int64_t M, int64_t, int64_t K) {
  return M <= int8_linear_max_rows(K) ? 0 : up256((size_t)(M * K)) + (size_t)M * 4;
}

hipError_t launch_int8_linear(const void* X, int xdtype, const float* act_scale, const void* W, const float* w_scales,
                              const float* bias, int64_t M, int64_t N, int64_t K, void* Y, void* workspace, hipStream_t stream) {
  if (M <= int8_linear_max_rows(K)) return launch_int8_linear_rows(X, xdtype, act_scale, W, w_scales, bias, M, N, K, Y, stream);
  float* const scales = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + up256((size_t)(M * K)));
  const hipError_t e = launch_int8_quantize(X, xdtype, act_scale, false, M, K, workspace, scales, stream);
  if (e != hipSuccess) return e;
  return launch_int8_gemm(workspace, scales, W, w_scales, bias, M, N, K, xdtype, Y, stream);
}

}  // namespace woq
