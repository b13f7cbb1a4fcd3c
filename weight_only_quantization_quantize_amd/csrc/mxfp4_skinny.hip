// Products of a few rows of activations with microscaled weights, or of more with
// few columns, bound by streaming the weights:
//   Y[m, n] = sum_b 2^(sA + sW - 254) sum_{k in block b} a[m, k] w[n, k].
//
// Work split.  K is cut into super-steps of 512 (four steps of 128).  A workgroup of 8
// waves holds `slots` teams of `team` waves; a wave owns one or two super-steps, whose
// activations stay in registers for the whole launch, and the team walks over its run
// of tiles of 16 columns of Y: the only traffic left is the weights'.  The team's
// partial sums of a tile meet in LDS and are added in a fixed order.  More rows than the
// registers hold (16 of 16-bit activations, 64 of 4-bit ones) are cut into row groups,
// workgroups of their own that read the same weights at the same time from the same L2.
//
// 16-bit activations are read from X as the matrix operands: a lane's part of a
// step is the 64 contiguous bytes of one block.
//
// Loads.  Units of 16 rows by 512 K in runs of 256 bytes (mxfp4_stream.h): loads
// of 16 rows x 64 bytes straight into the matrix operands reached 2.2 TB/s.  A wave
// has up to four units on their way, 139 KB a compute unit; 16 waves with one each
// had half of that and took 34 us for 16 rows of 28672 x 8192 (125 MB, 4-bit
// activations), where this takes 23; 16-bit ones take 32: the conversions and the
// longer matrix steps hold a unit's registers longer, and the loads wait for them.
#include "mxfp4_stream.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kWaves = 8;        // K <= 8192
constexpr int kLongWaves = 16;   // longer rows
constexpr int kTargetGroups = 256;  // workgroups: one per compute unit

// Activations: kMx, microscaled; kRows, 16-bit rows; kFragments, 16-bit ones laid out
// in fragments of 16 rows before (rows longer than the registers hold, read again for
// every tile).
enum Operand { kMx, kRows, kFragments };

// One super-step of a chunk of 16 rows of activations.
template <Operand OP>
struct Acts {
  MxActivations x;
};
template <>
struct Acts<kMx> {
  u32x4_t v[4];
  uint32_t s;
};

// Chunk t's super-step S; A, As, M: the row group's.
__device__ inline void load_acts(Acts<kMx>& act, const uint8_t* __restrict__ A, const uint8_t* __restrict__ As, int t, int S,
                                 int M, int nblk, int, int lane) {
  const int r = lane & 15, q = lane >> 4;
  int m = 16 * t + r;
  m = m < M ? m : M - 1;
  const int b0 = kSuper * S + 4 * q;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int b = b0 + s;
    const u32x4_t v = reinterpret_cast<const u32x4_t*>(A)[(uint32_t)(m * nblk + (b < nblk ? b : nblk - 1))];
    act.v[s] = b < nblk ? v : u32x4_t{0u, 0u, 0u, 0u};
  }
  const int from = b0 < nblk - 4 ? b0 : nblk - 4;  // a dword inside the row (K >= 128)
  __builtin_memcpy(&act.s, As + (uint32_t)(m * nblk + from), 4);
  act.s >>= 8 * ((b0 - from) & 3);
}
__device__ inline void load_acts(Acts<kRows>& act, const uint8_t* __restrict__ A, const uint8_t*, int t, int S, int M, int nblk,
                                 int, int lane) {
  int m = 16 * t + (lane & 15);
  m = m < M ? m : M - 1;
  mx_load_activations(act.x, reinterpret_cast<const uint16_t*>(A) + (int64_t)m * nblk * kMxBlock, nblk, S, lane);
}
__device__ inline void load_acts(Acts<kFragments>& act, const uint8_t* __restrict__ A, const uint8_t*, int t, int S, int, int,
                                 int supers, int lane) {
  mx_load_fragments(act.x, A + ((int64_t)t * supers + S) * 4 * kMxFragBytes, 16u * (uint32_t)lane);
}

// acc[t] += a staged unit of weights times chunk t's super-step of activations, of(t).
template <class XT, Operand OP, int TC, class F>
__device__ __forceinline__ void multiply(float4_t (&acc)[TC], F&& of, const uint8_t* __restrict__ stage, int lane) {
  if constexpr (OP == kMx) {
    const int scale = (int)mx_staged_scale(stage, lane);
    mx_each_step([&](auto sel) {
      constexpr int s = decltype(sel)::value;
      const i32x8_t w = mx_operand(mx_staged_weights(stage, s, lane));
#pragma unroll
      for (int t = 0; t < TC; ++t)
        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(of(t).v[s]), w, acc[t], kMfmaFp4, kMfmaFp4, s,
                                                                  (int)of(t).s, s, scale);
    });
  } else {
    static_assert(TC == 1, "16 rows");
    mx_multiply_unit<XT>(acc[0], of(0).x, stage, lane);
  }
}
// What the sums of products are multiplied by.
template <class XT, Operand OP>
constexpr float kGain = OP == kMx ? 1.0f : kMxGain<XT>;

// What a row group's workgroups see of the operands.
template <Operand OP, int TC>
__device__ inline void enter_row_group(const uint8_t* __restrict__& A, const uint8_t* __restrict__& As, int& M,
                                       uint16_t* __restrict__& Y, int N, int nblk, int supers) {
  const int m0 = (int)blockIdx.y * 16 * TC;
  M = M - m0 < 16 * TC ? M - m0 : 16 * TC;
  Y += (int64_t)m0 * N;
  if constexpr (OP == kMx) {
    A += (int64_t)m0 * nblk * 16;
    As += (int64_t)m0 * nblk;
  } else if constexpr (OP == kRows) {
    A += (int64_t)m0 * nblk * (2 * kMxBlock);
  } else {
    A += (int64_t)blockIdx.y * TC * supers * 4 * kMxFragBytes;
  }
}

// Rows 4 q .. 4 q + 3 of chunk t, column n of Y.
template <class YT>
__device__ inline void store(uint16_t* __restrict__ Y, int M, int N, int t, int n, int q, const float4_t& v, float gain) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int m = 16 * t + 4 * q + e;
    if (m < M && n < N) Y[(int64_t)m * N + n] = YT::from_f32(v[e] * gain);
  }
}

// K <= 8192.  A team's wave owns SU super-steps (tw, tw + team) whose activations
// stay in registers; the team takes TI tiles at a time while the next ones' units
// are on their way.
template <class YT, Operand OP, int TC, int SU, int TI>
__global__ __launch_bounds__(kWaves * 64, 2) void mxfp4_skinny_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ As, const uint8_t* __restrict__ W,
    const uint8_t* __restrict__ Ws, int M, int N, int nblk, int team, int supers, uint16_t* __restrict__ Y) {
  constexpr int NU = SU * TI;  // units a turn
  constexpr int kBuffers = TI * TC > 4 ? 1 : 2;
  __shared__ __attribute__((aligned(16))) uint8_t stage_all[kWaves][kUnitStage];
  __shared__ float4_t part[kBuffers][kWaves][TI * TC][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slots = (int)(blockDim.x >> 6) / team;
  const int slot = wave / team, tw = wave % team;
  uint8_t* const stage = stage_all[wave];
  enter_row_group<OP, TC>(A, As, M, Y, N, nblk, supers);

  // the team's run of tiles; all teams of the workgroup make as many turns
  const int tiles = (N + 15) >> 4, teams = (int)gridDim.x * slots;
  auto run = [&](int g) { return (int)((int64_t)tiles * g / teams); };
  const int begin = run((int)blockIdx.x * slots + slot), end = run((int)blockIdx.x * slots + slot + 1);
  int longest = 0;
  for (int g = 0; g < slots; ++g) {
    const int n = run((int)blockIdx.x * slots + g + 1) - run((int)blockIdx.x * slots + g);
    longest = n > longest ? n : longest;
  }

  auto super_of = [&](int j) { return tw + j % SU * team; };
  MxUnit u[NU];
  auto ahead = [&](int j, int t0) {
    const int tile = t0 + j / SU, S = super_of(j);
    const bool live = tile < end && S < supers;  // else a line or two in its place
    const int64_t row = live ? (int64_t)tile * 16 : 0;
    __builtin_amdgcn_sched_barrier(0);
    mx_load_unit(u[j], W + row * nblk * 16, Ws + row * nblk, (int)(N - row - 1), (N - row) * nblk, live ? nblk : 1, live ? S : 0, lane);
    __builtin_amdgcn_sched_barrier(0);
  };
  Acts<OP> act[TC][SU];
#pragma unroll
  for (int t = 0; t < TC; ++t)
#pragma unroll
    for (int i = 0; i < SU; ++i)
      load_acts(act[t][i], A, As, t, super_of(i) < supers ? super_of(i) : supers - 1, M, nblk, supers, lane);
  // (before the activations instead: 4-bit products took 1 .. 1.5 us more)
#pragma unroll
  for (int j = 0; j < NU; ++j) ahead(j, begin);
  if constexpr (OP == kRows) {  // while the weights come
#pragma unroll
    for (int t = 0; t < TC; ++t)
#pragma unroll
      for (int i = 0; i < SU; ++i) mx_mask_activations(act[t][i].x, nblk, super_of(i), lane);
  }
  float4_t acc[TI][TC];
  auto take = [&](int t0, auto more) {
    int l = lane;
    asm volatile("" : "+v"(l));  // LDS addresses are worked out each turn: kept, they spill
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const int tile = t0 + j / SU, S = super_of(j);
      const int64_t row = (int64_t)tile * 16;
      const bool live = tile < end && S < supers;
      if (live) mx_stage_unit(u[j], stage, (int)(N - row - 1), (N - row) * nblk, nblk, S, l);
      if constexpr (decltype(more)::value) ahead(j, t0 + TI);
      if (live) multiply<YT, OP>(acc[j / SU], [&](int t) -> const Acts<OP>& { return act[t][j % SU]; }, stage, l);
    }
  };
  const int turns = (longest + TI - 1) / TI;
  for (int it = 0; it < turns; ++it) {
    const int t0 = begin + it * TI;
#pragma unroll
    for (int i = 0; i < TI * TC; ++i) acc[i / TC][i % TC] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (it + 1 < turns)
      take(t0, std::true_type{});
    else
      take(t0, std::false_type{});
    float4_t(*const sums)[TI * TC][64] = part[kBuffers == 2 ? it & 1 : 0];
#pragma unroll
    for (int i = 0; i < TI * TC; ++i) sums[wave][i][lane] = acc[i / TC][i % TC];
    __syncthreads();
    // a wave adds the team's partials of a tile and chunk, in order, other waves each turn
    int l = lane;
    asm volatile("" : "+v"(l));
#pragma unroll
    for (int i = 0; i < TI * TC; ++i) {
      const int tile = t0 + i / TC;
      if (tile < end && tw == (it * TI * TC + i) % team) {
        float4_t v = sums[slot * team][i][l];
        for (int w = 1; w < team; ++w) {
          const float4_t p = sums[slot * team + w][i][l];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += p[e];
        }
        store<YT>(Y, M, N, i % TC, tile * 16 + (l & 15), l >> 4, v, kGain<YT, OP>);
      }
    }
    if (kBuffers == 1) __syncthreads();
  }
}

// Longer rows: wave w takes the super-steps w, w + 16, ... of a tile and loads the
// activations of each; the next unit is on its way meanwhile.
template <class YT, Operand OP, int TC>
__global__ __launch_bounds__(kLongWaves * 64) void mxfp4_skinny_long_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ As, const uint8_t* __restrict__ W,
    const uint8_t* __restrict__ Ws, int M, int N, int nblk, int supers, uint16_t* __restrict__ Y) {
  constexpr int team = kLongWaves;
  __shared__ __attribute__((aligned(16))) uint8_t stage_all[team][kUnitStage];
  __shared__ float4_t part[2][team][TC][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = (N + 15) >> 4;
  uint8_t* const stage = stage_all[wave];
  enter_row_group<OP, TC>(A, As, M, Y, N, nblk, supers);

  MxUnit u;
  auto left = [&](int tile) { return (int64_t)(N - tile * 16) * nblk; };  // scale bytes from the tile on
  auto load_weights = [&](int tile, int S) {
    mx_load_unit(u, W + (int64_t)tile * 16 * nblk * 16, Ws + (int64_t)tile * 16 * nblk, N - tile * 16 - 1, left(tile), nblk, S, lane);
  };
  // every wave makes the same number of turns; one without a super-step multiplies nothing
  const int rounds = (supers + team - 1) / team;
  int tile = blockIdx.x;
  load_weights(tile, wave);
  for (int it = 0; tile < tiles; ++it) {
    const int next = tile + (int)gridDim.x;
    float4_t acc[TC] = {};
    for (int k = 0; k < rounds; ++k) {
      const int S = wave + k * team;
      int l = lane;
      if constexpr (OP == kFragments) asm volatile("" : "+v"(l));  // addresses are worked out each time: kept, they spill
      mx_stage_unit(u, stage, N - tile * 16 - 1, left(tile), nblk, S, l);
      Acts<OP> act[TC];
#pragma unroll
      for (int t = 0; t < TC; ++t) load_acts(act[t], A, As, t, S < supers ? S : supers - 1, M, nblk, supers, l);
      const int Sn = k + 1 < rounds ? S + team : wave;
      const int tn = k + 1 < rounds ? tile : next;
      load_weights(tn < tiles ? tn : tile, Sn < supers ? Sn : supers - 1);
      if (S < supers) multiply<YT, OP>(acc, [&](int t) -> const Acts<OP>& { return act[t]; }, stage, l);
    }
    const int buf = it & 1;
    int l = lane;
    if constexpr (OP == kFragments) asm volatile("" : "+v"(l));
#pragma unroll
    for (int t = 0; t < TC; ++t) part[buf][wave][t][l] = acc[t];
    __syncthreads();
    // a wave a chunk adds the partials, other ones each turn
#pragma unroll
    for (int t = 0; t < TC; ++t) {
      if (wave == (it + t) % team) {
        float4_t v = part[buf][0][t][l];
        for (int w = 1; w < team; ++w) {
          const float4_t p = part[buf][w][t][l];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += p[e];
        }
        store<YT>(Y, M, N, t, tile * 16 + (l & 15), l >> 4, v, kGain<YT, OP>);
      }
    }
    tile = next;
  }
}

// Workgroups a row group: a multiple of 8, so that a column group's are on one XCD
// (three row groups of 85 took 28 us where four of 64 take 26).
int share(int rgroups) {
  const int n = kTargetGroups / rgroups & ~7;
  return n < 8 ? 8 : n;
}

template <class YT, Operand OP, int TC>
hipError_t launch_long(const void* A, const void* As, const void* W, const void* Ws, int M, int N, int nblk, void* Y,
                       hipStream_t stream) {
  const int tiles = (N + 15) / 16, rgroups = (M + 16 * TC - 1) / (16 * TC), target = share(rgroups);
  const dim3 grid((unsigned)(tiles < target ? tiles : target), (unsigned)rgroups);
  mxfp4_skinny_long_kernel<YT, OP, TC><<<grid, kLongWaves * 64, 0, stream>>>(
      static_cast<const uint8_t*>(A), static_cast<const uint8_t*>(As), static_cast<const uint8_t*>(W),
      static_cast<const uint8_t*>(Ws), M, N, nblk, (nblk + kSuper - 1) / kSuper, static_cast<uint16_t*>(Y));
  return hipGetLastError();
}

template <class YT, Operand OP, int TC>
hipError_t launch(const void* A, const void* As, const void* W, const void* Ws, int M, int N, int nblk, void* Y,
                  hipStream_t stream) {
  const int tiles = (N + 15) / 16, supers = (nblk + kSuper - 1) / kSuper;
  const int rgroups = (M + 16 * TC - 1) / (16 * TC), target = share(rgroups);
  if constexpr (OP == kMx && TC < 4)  // 64 rows at once come with K <= 8192 only
    if (supers > 2 * kWaves) return launch_long<YT, OP, TC>(A, As, W, Ws, M, N, nblk, Y, stream);
  const bool two = supers > kWaves;
  const int team = two ? (supers + 1) / 2 : supers;
  // short rows: several teams a workgroup, where there are tiles for them
  int slots = kWaves / team;
  const int per = (tiles + target - 1) / target;
  slots = slots < per ? slots : per;
  const int groups = (tiles + slots - 1) / slots;
  const dim3 grid((unsigned)(groups < target ? groups : target), (unsigned)rgroups);
  // four units ahead (16 rows of 16384 x 4096: 13.7 us, with one 15), fewer where a team
  // has fewer tiles (units that are not there cost their loads all the same: 4096 x
  // 4096 takes 8.2 us with one, 9.9 with four) or where 64 rows leave no registers for
  // them
  const int most = (tiles + (int)grid.x * slots - 1) / ((int)grid.x * slots);
  auto* const f = [&] {
    if constexpr (TC == 4)  // N > 8192: several tiles a team
      return two ? mxfp4_skinny_kernel<YT, kMx, 4, 2, 1> : mxfp4_skinny_kernel<YT, kMx, 4, 1, 2>;
    else
      return two ? (most > 1 ? mxfp4_skinny_kernel<YT, OP, TC, 2, 2> : mxfp4_skinny_kernel<YT, OP, TC, 2, 1>)
                 : (most > 2   ? mxfp4_skinny_kernel<YT, OP, TC, 1, 4>
                    : most > 1 ? mxfp4_skinny_kernel<YT, OP, TC, 1, 2>
                               : mxfp4_skinny_kernel<YT, OP, TC, 1, 1>);
  }();
  f<<<grid, (unsigned)(slots * team * 64), 0, stream>>>(static_cast<const uint8_t*>(A), static_cast<const uint8_t*>(As),
                                                        static_cast<const uint8_t*>(W), static_cast<const uint8_t*>(Ws), M, N,
                                                        nblk, team, supers, static_cast<uint16_t*>(Y));
  return hipGetLastError();
}

}  // namespace

// 16-bit activations: rows of X (K <= mxfp4_skinny_max_k()), or fragments of 16 rows.
int64_t mxfp4_skinny_max_k() { return 2 * kWaves * 512; }
hipError_t launch_mxfp4_skinny(const void* X, int xdtype, const void* codes, const void* scales, int64_t M, int64_t N, int64_t K,
                               void* Y, hipStream_t stream) {
  const int nblk = (int)(K / kMxBlock);
  auto* const f = K <= mxfp4_skinny_max_k() ? (xdtype == 0 ? launch<F16, kRows, 1> : launch<BF16, kRows, 1>)
                                            : (xdtype == 0 ? launch_long<F16, kFragments, 1> : launch_long<BF16, kFragments, 1>);
  return f(X, nullptr, codes, scales, (int)M, (int)N, nblk, Y, stream);
}

// Microscaled activations.
hipError_t launch_mxfp4_skinny_mx(const void* A, const void* As, const void* codes, const void* scales, int64_t M,
                                  int64_t N, int64_t K, int ydtype, void* Y, hipStream_t stream) {
  const int nblk = (int)(K / kMxBlock);
  // chunks of 16 rows a workgroup: all of them, so that the weights are read once,
  // but two where there are few columns and a workgroup would load more activations
  // than weights (64 rows of 4096 x 4096: 6.6 us in two row groups, 8.0 in one;
  // 28672 x 8192: 34, 31)
  const int chunks = M <= 16 ? 1 : (M <= 32 || N <= 8192 ? 2 : 4);
  auto* const f = chunks == 1   ? (ydtype == 0 ? launch<F16, kMx, 1> : launch<BF16, kMx, 1>)
                  : chunks == 2 ? (ydtype == 0 ? launch<F16, kMx, 2> : launch<BF16, kMx, 2>)
                                : (ydtype == 0 ? launch<F16, kMx, 4> : launch<BF16, kMx, 4>);
  return f(A, As, codes, scales, (int)M, (int)N, nblk, Y, stream);
}

}  // namespace woq
