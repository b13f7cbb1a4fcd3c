// Matrix products with a microscaled 4-bit right operand W [N, K]:
//   PIECES = 1: a microscaled 4-bit left operand A [M, K], both as stored;
//   PIECES = 3: 16-bit activations split into three 6-bit pieces
//               (mxfp4_split_kernel; mxfp4_device.h says why).
// Y[m, n] = sum over the 32-element blocks b of 2^(sA + sW - 254) sum_k a w,
// all of it inside v_mfma_scale_f32_32x32x64_f8f6f4: no element is decoded,
// the products are exact and the sums are the matrix unit's fp32.
//
// A workgroup of 2 x 2 waves computes 64 TM x 64 TN of Y in K tiles of 128,
// double-buffered in LDS by direct loads (16 bytes a lane).
//
// LDS layout of a 4-bit operand: a row's 64 bytes of a K tile are four chunks
// of one block each, chunk c at position c ^ ((row / 4) % 4), so that the 16
// rows a quarter wave reads at one chunk lie in 16 different 16-byte slots of
// the 256-byte bank row.
#include "mxfp4_device.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kBK = 128;              // K per tile
constexpr int kRowBytes = kBK / 2;    // of a 4-bit operand
constexpr int kThreads = 256;

typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void glb_void;

// 64 lanes x 16 bytes from per-lane addresses to consecutive LDS.
__device__ inline void load_to_lds(const void* g, void* l) {
  __builtin_amdgcn_global_load_lds((glb_void*)g, (lds_void*)l, 16, 0, 0);
}

template <class YT, int PIECES, int TM, int TN>
__global__ __launch_bounds__(kThreads) void mxfp4_gemm_kernel(const uint8_t* __restrict__ A,
                                                              const uint8_t* __restrict__ As,
                                                              const uint8_t* __restrict__ W,
                                                              const uint8_t* __restrict__ Ws, int M, int N, int K,
                                                              uint16_t* __restrict__ Y) {
  constexpr int BM = 64 * TM, BN = 64 * TN;
  constexpr int kABytes = PIECES == 1 ? BM * kRowBytes : BM / 32 * 2 * kMxFragBytes;
  constexpr int kBBytes = BN * kRowBytes;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][kABytes + kBBytes];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int half = lane >> 5, r32 = lane & 31;
  const int nblk = K / kMxBlock, ktiles = (K + kBK - 1) / kBK;
  const int m0 = (int)blockIdx.x * BM, n0 = (int)blockIdx.y * BN;

  // 4-bit operand tile: load j of a wave covers 16 rows, four lanes a row.
  auto issue4 = [&](const uint8_t* P, int row0, int rows, int tile_rows, int kt, uint8_t* dst) {
    const int sub = lane >> 2, pos = lane & 3;
#pragma unroll
    for (int j = 0; j < tile_rows / 64; ++j) {
      const int lr = (4 * j + wave) * 16 + sub;
      int r = row0 + lr;
      r = r < rows ? r : rows - 1;
      int c = 4 * kt + (pos ^ ((lr >> 2) & 3));
      c = c < nblk ? c : nblk - 1;  // past the row's end: any block, its partner operand is zeroed
      load_to_lds(P + ((int64_t)r * nblk + c) * 16, dst + (4 * j + wave) * 1024);
    }
  };
  auto issue = [&](int kt, int buf) {
    uint8_t* const a = lds[buf];
    if constexpr (PIECES == 1) {
      issue4(A, m0, M, BM, kt, a);
    } else {
      // per 32 rows 2 fragments = 9 loads of 1 KB
      constexpr int kLoads = BM / 32 * 9;
      for (int j = wave; j < kLoads; j += kThreads / 64) {
        const int rg = j / 9, part = j % 9;
        const int64_t f = (int64_t)(m0 / 32 + rg) * (2 * ktiles) + 2 * kt;
        load_to_lds(A + f * kMxFragBytes + part * 1024 + lane * 16, a + j * 1024);
      }
    }
    issue4(W, n0, N, BN, kt, a + kABytes);
  };
  uint32_t sa[2][TM * (PIECES == 1 ? 1 : 2)], sb[2][TN];
  auto issue_scales = [&](int kt, uint32_t* a, uint32_t* b) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      if constexpr (PIECES == 1) {
        int r = m0 + (wm * TM + i) * 32 + r32;
        r = r < M ? r : M - 1;
        a[i] = mx_load_scales(As + (int64_t)r * nblk, 4 * kt, nblk);
      } else {
        const int64_t f = (int64_t)(m0 / 32 + wm * TM + i) * (2 * ktiles) + 2 * kt;
        a[2 * i] = reinterpret_cast<const uint32_t*>(As)[f * 64 + lane];
        a[2 * i + 1] = reinterpret_cast<const uint32_t*>(As)[f * 64 + 64 + lane];
      }
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      int r = n0 + (wn * TN + j) * 32 + r32;
      r = r < N ? r : N - 1;
      b[j] = mx_load_scales(Ws + (int64_t)r * nblk, 4 * kt, nblk);
    }
  };

  float16_t acc[TM][TN] = {};
  auto frag4 = [&](const uint8_t* base, int row, int s) {
    const int c = (2 * s + half) ^ ((row >> 2) & 3);
    return *reinterpret_cast<const u32x4_t*>(base + row * kRowBytes + c * 16);
  };
  auto compute = [&](int kt, int buf, const uint32_t* a, const uint32_t* b) {
    const uint8_t* const la = lds[buf];
    const uint8_t* const lb = la + kABytes;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      // lane (row, half) multiplies block 2 s + half of its row
      i32x8_t bf[TN];
      int bs[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        bf[j] = mx_operand(frag4(lb, (wn * TN + j) * 32 + r32, s));
        bs[j] = (int)(b[j] >> (8 * (2 * s + half)));
      }
      if constexpr (PIECES == 1) {
        const bool live = 4 * kt + 2 * s + half < nblk;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          u32x4_t v = frag4(la, (wm * TM + i) * 32 + r32, s);
          v = live ? v : u32x4_t{0u, 0u, 0u, 0u};
          const int as = (int)(a[i] >> (8 * (2 * s + half)));
          const i32x8_t af = mx_operand(v);
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(af, bf[j], acc[i][j], kMfmaFp4, kMfmaFp4, 0, as, 0, bs[j]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const uint8_t* const fr = la + ((wm * TM + i) * 2 + s) * kMxFragBytes;
          const int as = (int)a[2 * i + s];
          auto piece = [&](int p) {
            return mx_operand(*reinterpret_cast<const u32x4_t*>(fr + p * kMxPieceBytes + 16 * lane),
                              *reinterpret_cast<const u32x2_t*>(fr + p * kMxPieceBytes + 1024 + 8 * lane));
          };
          // smallest piece first
          const i32x8_t p2 = piece(2), p1 = piece(1), p0 = piece(0);
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(p2, bf[j], acc[i][j], kMfmaFp6, kMfmaFp4, 2, as, 0, bs[j]);
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(p1, bf[j], acc[i][j], kMfmaFp6, kMfmaFp4, 1, as, 0, bs[j]);
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(p0, bf[j], acc[i][j], kMfmaFp6, kMfmaFp4, 0, as, 0, bs[j]);
        }
      }
    }
  };

  issue(0, 0);
  issue_scales(0, sa[0], sb[0]);
  __syncthreads();
  int kt = 0;
  for (; kt + 1 < ktiles; kt += 2) {
    issue(kt + 1, 1);
    issue_scales(kt + 1, sa[1], sb[1]);
    compute(kt, 0, sa[0], sb[0]);
    __syncthreads();
    if (kt + 2 < ktiles) {
      issue(kt + 2, 0);
      issue_scales(kt + 2, sa[0], sb[0]);
    }
    compute(kt + 1, 1, sa[1], sb[1]);
    __syncthreads();
  }
  if (kt < ktiles) compute(kt, 0, sa[0], sb[0]);

  // D: lane holds column r32, rows 8 (i / 4) + 4 half + i % 4.
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int n = n0 + (wn * TN + j) * 32 + r32;
      if (n < N) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int m = m0 + (wm * TM + i) * 32 + 8 * (e >> 2) + 4 * half + (e & 3);
          if (m < M) Y[(int64_t)m * N + n] = YT::from_f32(acc[i][j][e]);
        }
      }
    }
}

template <class YT, int PIECES>
hipError_t launch(const void* A, const void* As, const void* W, const void* Ws, int64_t M, int64_t N, int64_t K,
                  void* Y, hipStream_t stream) {
  constexpr int TM = 2, TN = 2;
  const dim3 grid((unsigned)((M + 64 * TM - 1) / (64 * TM)), (unsigned)((N + 64 * TN - 1) / (64 * TN)));
  mxfp4_gemm_kernel<YT, PIECES, TM, TN><<<grid, kThreads, 0, stream>>>(
      static_cast<const uint8_t*>(A), static_cast<const uint8_t*>(As), static_cast<const uint8_t*>(W),
      static_cast<const uint8_t*>(Ws), (int)M, (int)N, (int)K, static_cast<uint16_t*>(Y));
  return hipGetLastError();
}

constexpr int64_t kSkinnyRows = 64;     // up to here the weight-streaming kernel, 16-bit activations
constexpr int64_t kSkinnyRowsMx = 64;   // and microscaled ones
bool skinny(int64_t M, int64_t K, int64_t rows) { return M <= rows && K >= 128; }
constexpr int64_t kRowPad = 128;  // rows of split activations are padded to a tile

int64_t split_row_groups(int64_t M) { return (M + kRowPad - 1) / kRowPad * (kRowPad / 32); }
int64_t split_ksteps(int64_t K) { return (K + kBK - 1) / kBK * 2; }

}  // namespace

size_t mxfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M == 1 && K <= mxfp4_gemv_max_k()) return 0;
  if (skinny(M, K, kSkinnyRows)) return (size_t)((M + 15) / 16 * ((K + 511) / 512 * 4)) * (kMxFragBytes + kMxFragScaleBytes);
  return (size_t)(split_row_groups(M) * split_ksteps(K)) * (kMxFragBytes + kMxFragScaleBytes);
}

hipError_t launch_mxfp4_gemm(const void* X, int xdtype, const void* codes, const void* scales, int64_t M, int64_t N,
                             int64_t K, void* Y, void* workspace, hipStream_t stream) {
  if (M == 1 && K <= mxfp4_gemv_max_k()) return launch_mxfp4_gemv(X, xdtype, codes, scales, N, K, Y, stream);
  uint8_t* const pieces = static_cast<uint8_t*>(workspace);
  if (skinny(M, K, kSkinnyRows)) {
    const int64_t steps = (K + 511) / 512 * 4, groups = (M + 15) / 16;
    uint8_t* const ps = pieces + groups * steps * kMxFragBytes;
    const hipError_t e = launch_mxfp4_split(X, xdtype, M, K, 16, groups, steps, pieces, ps, stream);
    if (e != hipSuccess) return e;
    return launch_mxfp4_skinny(pieces, ps, codes, scales, M, N, K, xdtype, Y, stream);
  }
  const int64_t rg = split_row_groups(M), ks = split_ksteps(K);
  uint8_t* const ps = pieces + rg * ks * kMxFragBytes;
  const hipError_t e = launch_mxfp4_split(X, xdtype, M, K, 32, rg, ks, pieces, ps, stream);
  if (e != hipSuccess) return e;
  return xdtype == 0 ? launch<F16, kMxPieces>(pieces, ps, codes, scales, M, N, K, Y, stream)
                     : launch<BF16, kMxPieces>(pieces, ps, codes, scales, M, N, K, Y, stream);
}

hipError_t launch_mxfp4_gemm_mx(const void* A, const void* As, const void* W, const void* Ws, int64_t M, int64_t N,
                                int64_t K, int ydtype, void* Y, hipStream_t stream) {
  if (skinny(M, K, kSkinnyRowsMx)) return launch_mxfp4_skinny_mx(A, As, W, Ws, M, N, K, ydtype, Y, stream);
  return ydtype == 0 ? launch<F16, 1>(A, As, W, Ws, M, N, K, Y, stream) : launch<BF16, 1>(A, As, W, Ws, M, N, K, Y, stream);
}

}  // namespace woq
