// Products of a few rows of activations with microscaled weights (2 to 16 rows
// of 16-bit activations, up to 64 rows of microscaled ones), bound by
// streaming the weights:
//   Y[m, n] = sum_b 2^(sA + sW - 254) sum_{k in block b} a[m, k] w[n, k].
//
// Work split.  K is cut into super-steps of 512 (four steps of
// v_mfma_scale_f32_16x16x128).  A workgroup holds `slots` teams of `team` waves;
// wave w of a team owns the super-steps w, w + team, ... and the team walks over
// tiles of 16 columns of Y.  Up to K = 8192 a wave owns one super-step and its
// activations stay in registers for the whole launch (RESIDENT); the only
// traffic left is the weights'.  The team's partial sums of a tile meet in LDS
// and are added in a fixed order.  More rows than the registers hold (16 of
// three pieces, 32 of 4-bit activations) are cut into row groups, workgroups
// of their own that read the same weights at the same time from the same L2 (a
// column group's lie a multiple of 8 apart in dispatch order).
//
// Loads.  Units of 16 rows by 512 K in runs of 256 bytes (mxfp4_stream.h): loads
// of 16 rows x 64 bytes straight into the matrix operands reached 2.2 TB/s.  The
// next unit is loaded as soon as this one is in LDS.
#include "mxfp4_stream.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kMaxWaves = 16;
constexpr int kMaxThreads = kMaxWaves * 64;
constexpr int kTargetGroups = 256;  // workgroups: one per compute unit

// One super-step of a chunk of 16 rows of activations.
template <int PIECES>
struct Acts;
template <>
struct Acts<1> {
  u32x4_t v[4];
  uint32_t s;
};
template <>
struct Acts<kMxPieces> {
  MxActivations a[4];
};

template <class YT, int PIECES, int TC, bool RESIDENT>
__global__ __launch_bounds__(kMaxThreads) void mxfp4_skinny_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ As, const uint8_t* __restrict__ W,
    const uint8_t* __restrict__ Ws, int M, int N, int nblk, int team, int supers, uint16_t* __restrict__ Y) {
  __shared__ __attribute__((aligned(16))) uint8_t stage_all[kMaxWaves][kUnitStage];
  __shared__ float4_t part[2][kMaxWaves][TC][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slots = (int)(blockDim.x >> 6) / team;
  const int slot = wave / team, tw = wave % team;
  const int r = lane & 15, q = lane >> 4;
  const int tiles = (N + 15) >> 4;
  uint8_t* const stage = stage_all[wave];
  // row group blockIdx.y: 16 TC rows
  const int m0 = (int)blockIdx.y * 16 * TC;
  M = M - m0 < 16 * TC ? M - m0 : 16 * TC;
  Y += (int64_t)m0 * N;
  if constexpr (PIECES == 1) {
    A += (int64_t)m0 * nblk * 16;
    As += (int64_t)m0 * nblk;
  } else {
    A += (int64_t)blockIdx.y * TC * supers * 4 * kMxFragBytes;
    As += (int64_t)blockIdx.y * TC * supers * 4 * kMxFragScaleBytes;
  }

  MxUnit u;
  auto left = [&](int tile) { return (int64_t)(N - tile * 16) * nblk; };  // scale bytes from the tile on
  auto load_weights = [&](int tile, int S) {
    mx_load_unit(u, W + (int64_t)tile * 16 * nblk * 16, Ws + (int64_t)tile * 16 * nblk, N - tile * 16 - 1, left(tile), nblk, S, lane);
  };
  Acts<PIECES> act[TC];
  auto load_acts = [&](int S) {
#pragma unroll
    for (int t = 0; t < TC; ++t) {
      if constexpr (PIECES == 1) {
        int m = 16 * t + r;
        m = m < M ? m : M - 1;
        const int b0 = kSuper * S + 4 * q;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int b = b0 + s;
          const u32x4_t v = reinterpret_cast<const u32x4_t*>(A)[(uint32_t)(m * nblk + (b < nblk ? b : nblk - 1))];
          act[t].v[s] = b < nblk ? v : u32x4_t{0u, 0u, 0u, 0u};
        }
        const int from = b0 < nblk - 4 ? b0 : nblk - 4;  // a dword inside the row (K >= 128)
        __builtin_memcpy(&act[t].s, As + (uint32_t)(m * nblk + from), 4);
        act[t].s >>= 8 * ((b0 - from) & 3);
      } else {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int64_t f = ((int64_t)t * supers + S) * 4 + s;
          mx_load_activations(act[t].a[s], A + f * kMxFragBytes, As + f * kMxFragScaleBytes, mx_place(0, lane));
        }
      }
    }
  };

  const int first = (int)blockIdx.x * slots + slot, step = (int)gridDim.x * slots;
  if constexpr (RESIDENT) load_acts(tw);
  int tile = first < tiles ? first : tiles - 1;  // teams past the last tile keep the barriers' company
  load_weights(tile, tw);
  // every team of the workgroup makes the same number of turns of the same
  // number of super-steps; a wave without one (K short of it) multiplies zeros
  const int turns = (tiles - (int)blockIdx.x * slots + step - 1) / step;
  const int per_turn = RESIDENT ? 1 : (supers + team - 1) / team;
  float4_t acc[TC] = {};
  for (int i = 0, it = 0, k = 0; i < turns * per_turn; ++i) {
    const int S = RESIDENT ? tw : tw + k * team;
    mx_stage_unit(u, stage, N - tile * 16 - 1, left(tile), nblk, S, lane);
    const bool wraps = RESIDENT || k + 1 == per_turn;
    const int next = wraps ? (tile + step < tiles ? tile + step : tiles - 1) : tile;
    if constexpr (!RESIDENT) load_acts(S < supers ? S : supers - 1);
    if (i + 1 < turns * per_turn) {
      const int Sn = RESIDENT || wraps ? tw : S + team;
      load_weights(next, Sn < supers ? Sn : supers - 1);
    }
    const int scale = mx_staged_scale(stage, lane);
    if (RESIDENT || S < supers) {
      mx_each_step([&](auto sel) {
        constexpr int s = decltype(sel)::value;
        const i32x8_t w = mx_staged_weights(stage, s, lane);
#pragma unroll
        for (int t = 0; t < TC; ++t) {
          if constexpr (PIECES == 1)
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(act[t].v[s]), w, acc[t], kMfmaFp4,
                                                                      kMfmaFp4, s, (int)act[t].s, s, scale);
          else
            mx_multiply<s>(acc[t], act[t].a[s], w, scale);
        }
      });
    }
    ++k;
    if (!wraps) continue;
    const int buf = it & 1;
#pragma unroll
    for (int t = 0; t < TC; ++t) part[buf][wave][t][lane] = acc[t];
    __syncthreads();
    // one wave a chunk adds the team's partials, another one each turn
    const bool live = first + it * step < tiles;
#pragma unroll
    for (int t = 0; t < TC; ++t) {
      if (live && tw == (it + t) % team) {
        float4_t v = part[buf][slot * team][t][lane];
        for (int w = 1; w < team; ++w) {
          const float4_t p = part[buf][slot * team + w][t][lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += p[e];
        }
        if (tile * 16 + r < N) {
          uint16_t* const yt = Y + (int64_t)tile * 16;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = 16 * t + 4 * q + e;
            if (m < M) yt[(uint32_t)(m * N + r)] = YT::from_f32(v[e]);
          }
        }
      }
      acc[t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    tile = next;
    ++it;
    k = 0;
  }
}

template <class YT, int PIECES, int TC>
hipError_t launch(const void* A, const void* As, const void* W, const void* Ws, int M, int N, int nblk, void* Y,
                  hipStream_t stream) {
  const auto* ap = static_cast<const uint8_t*>(A);
  const auto* asp = static_cast<const uint8_t*>(As);
  const auto* wp = static_cast<const uint8_t*>(W);
  const auto* wsp = static_cast<const uint8_t*>(Ws);
  auto* yp = static_cast<uint16_t*>(Y);
  const int tiles = (N + 15) / 16, supers = (nblk + kSuper - 1) / kSuper;
  const int team = supers < kMaxWaves ? supers : kMaxWaves;
  // short rows: several teams a workgroup, where there are tiles for them
  int slots = kMaxWaves / team;
  const int per = (tiles + kTargetGroups - 1) / kTargetGroups;
  slots = slots < per ? slots : per;
  const int groups = (tiles + slots - 1) / slots;
  const int rgroups = (M + 16 * TC - 1) / (16 * TC), target = kTargetGroups / rgroups;
  const dim3 grid((unsigned)(groups < target ? groups : target), (unsigned)rgroups);
  const unsigned threads = (unsigned)(slots * team * 64);
  if (supers <= kMaxWaves)
    mxfp4_skinny_kernel<YT, PIECES, TC, true><<<grid, threads, 0, stream>>>(ap, asp, wp, wsp, M, N, nblk, team, supers, yp);
  else
    mxfp4_skinny_kernel<YT, PIECES, TC, false><<<grid, threads, 0, stream>>>(ap, asp, wp, wsp, M, N, nblk, team, supers, yp);
  return hipGetLastError();
}

}  // namespace

// 16-bit activations, split in fragments of 16 rows.
hipError_t launch_mxfp4_skinny(const void* pieces, const void* piece_scales, const void* codes, const void* scales,
                               int64_t M, int64_t N, int64_t K, int ydtype, void* Y, hipStream_t stream) {
  const int nblk = (int)(K / kMxBlock);
  return ydtype == 0 ? launch<F16, kMxPieces, 1>(pieces, piece_scales, codes, scales, (int)M, (int)N, nblk, Y, stream)
                     : launch<BF16, kMxPieces, 1>(pieces, piece_scales, codes, scales, (int)M, (int)N, nblk, Y, stream);
}

// Microscaled activations.
hipError_t launch_mxfp4_skinny_mx(const void* A, const void* As, const void* codes, const void* scales, int64_t M,
                                  int64_t N, int64_t K, int ydtype, void* Y, hipStream_t stream) {
  const int nblk = (int)(K / kMxBlock);
  auto* const f = M <= 16 ? (ydtype == 0 ? launch<F16, 1, 1> : launch<BF16, 1, 1>)
                          : (ydtype == 0 ? launch<F16, 1, 2> : launch<BF16, 1, 2>);
  return f(A, As, codes, scales, (int)M, (int)N, nblk, Y, stream);
}

}  // namespace woq
