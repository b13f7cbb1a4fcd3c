// GEMV with microscaled 4-bit weights for one row of 16-bit activations:
//   y[n] = sum_b 2^(s[n,b] - 127) sum_{k in block b} x[k] w[n,k].
//
// Bound by streaming the codes and scales once: 17/32 byte per weight.  A lane
// owns one block of 32 K (16 bytes of codes, one scale byte); its 32
// activations stay in 16 registers while rows stream past.  A code pair is
// widened to the activation's type by one conversion at a fixed scale, where every
// e2m1 value is exact, and multiplied by one dot2 with fp32 accumulation; the
// block's sum is then scaled in fp32, so no weight is rounded whatever its scale
// and x is used as given.  The fixed scale is 1 for fp16 (a block's sum is below
// 2^24) and 2^-8 for bf16: 32 products of up to 6 2^-8 2^128 stay below 2^128, and
// those of bf16's smallest number 2^-133 are multiples of 2^-142, which fp32 holds.
//
// Rows.  A row's blocks are spread over `team` lanes (a power of two up to 64;
// longer rows over several waves, `segs` of them).  A workgroup holds 8 waves
// (fewer where segs does not divide 8) and STEPS row steps with all their
// loads in flight at once; workgroup b takes row groups b, b + B, ..., so the
// whole GPU reads one window of rows at a time.  The lanes' partial sums meet
// in LDS after the stream, one reduction for all steps.
#include "mxfp4_device.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kWaves = 8;
constexpr int kMaxSegs = 8;  // K <= 8 * 64 * 32 = 16384 here

// sum of x times the weights of scale byte b
template <class XT>
__device__ inline float block_dot(u32x4_t c, const uint32_t (&x)[16], uint32_t b) {
  float p = 0.0f, q = 0.0f;
  constexpr float kScale = kMxIsF16<XT> ? 1.0f : 0x1p-8f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const u32x4_t w = mx_widen_as_is<XT>(c[j], __builtin_bit_cast(uint32_t, kScale) >> 23);
    p = XT::dot2(w[0], x[4 * j], p);
    q = XT::dot2(w[1], x[4 * j + 1], q);
    p = XT::dot2(w[2], x[4 * j + 2], p);
    q = XT::dot2(w[3], x[4 * j + 3], q);
  }
  if constexpr (kMxIsF16<XT>) return (p + q) * mx_pow2(b);
  const float d = ldexpf(p + q, (int)b - 127 + 8);  // 2^(b - 119) itself may be out of range
  return b == (uint32_t)kMxNan ? __builtin_bit_cast(float, 0x7FC00000u) : d;
}

// nblk: blocks per row.  Thread layout: wave = slot * segs + seg; a wave holds
// 64 / team rows.
template <class XT, int STEPS>
__global__ __launch_bounds__(kWaves * 64) void mxfp4_gemv_kernel(const uint16_t* __restrict__ x,
                                                                 const uint8_t* __restrict__ codes,
                                                                 const uint8_t* __restrict__ scales, int N, int nblk,
                                                                 int segs, int team, uint16_t* __restrict__ y) {
  __shared__ float part[STEPS][kWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int seg = wave % segs, slot = wave / segs, slots = (int)(blockDim.x >> 6) / segs;
  const int rpw = 64 / team;                     // rows per wave
  const int rows = slots * rpw;                  // rows per workgroup and step
  const int blk = 64 * seg + lane % team;        // this lane's block (64 lanes per row where segs > 1)
  const bool live = blk < nblk;
  const int cb = live ? blk : nblk - 1;          // clamped: loads stay inside the row
  const int row0 = (int)blockIdx.x * rows + slot * rpw + lane / team;
  const int stride = (int)gridDim.x * rows;

  uint32_t xr[16];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const u32x4_t v = reinterpret_cast<const u32x4_t*>(x)[4 * cb + q];
#pragma unroll
    for (int e = 0; e < 4; ++e) xr[4 * q + e] = live ? v[e] : 0u;
  }
  u32x4_t c[STEPS];
  uint32_t s[STEPS];
#pragma unroll
  for (int st = 0; st < STEPS; ++st) {
    const int r = row0 + st * stride;
    const int64_t at = (int64_t)(r < N ? r : N - 1) * nblk + cb;
    c[st] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(codes) + at);
    s[st] = scales[at];
  }
#pragma unroll
  for (int st = 0; st < STEPS; ++st) {
    const float d = block_dot<XT>(c[st], xr, s[st]);
    part[st][wave][lane] = live ? d : 0.0f;
  }
  __syncthreads();
  // one (step, slot) of outputs per wave at a time: the segments' partials,
  // then the team's lanes
  for (int o = wave; o < STEPS * slots; o += (int)(blockDim.x >> 6)) {
    const int st = o / slots, sl = o % slots;
    float v = 0.0f;
    for (int g = 0; g < segs; ++g) v += part[st][sl * segs + g][lane];
    v = team_sum(v, team);
    const int r = (int)blockIdx.x * rows + sl * rpw + lane / team + st * stride;
    if (lane % team == 0 && r < N) y[r] = XT::from_f32(v);
  }
}

template <class XT>
hipError_t launch(const void* x, const void* codes, const void* scales, int N, int nblk, void* y, hipStream_t stream) {
  const int segs = (nblk + 63) / 64;
  int team = 64;
  if (segs == 1)
    while (team > 1 && team / 2 >= nblk) team /= 2;
  const int slots = kWaves / segs;
  const int rows = slots * (64 / team);
  const int groups = (N + rows - 1) / rows;
  const dim3 block((unsigned)(slots * segs * 64));
  const auto* xp = static_cast<const uint16_t*>(x);
  const auto* cp = static_cast<const uint8_t*>(codes);
  const auto* sp = static_cast<const uint8_t*>(scales);
  auto* yp = static_cast<uint16_t*>(y);
  // as many row steps as still leave two workgroups per compute unit
  if (groups >= 2048)
    mxfp4_gemv_kernel<XT, 4><<<(unsigned)((groups + 3) / 4), block, 0, stream>>>(xp, cp, sp, N, nblk, segs, team, yp);
  else if (groups >= 1024)
    mxfp4_gemv_kernel<XT, 2><<<(unsigned)((groups + 1) / 2), block, 0, stream>>>(xp, cp, sp, N, nblk, segs, team, yp);
  else
    mxfp4_gemv_kernel<XT, 1><<<(unsigned)groups, block, 0, stream>>>(xp, cp, sp, N, nblk, segs, team, yp);
  return hipGetLastError();
}

}  // namespace

int64_t mxfp4_gemv_max_k() { return (int64_t)kMaxSegs * 64 * kMxBlock; }

hipError_t launch_mxfp4_gemv(const void* x, int xdtype, const void* codes, const void* scales, int64_t N, int64_t K,
                             void* y, hipStream_t stream) {
  return xdtype == 0 ? launch<F16>(x, codes, scales, (int)N, (int)(K / kMxBlock), y, stream)
                     : launch<BF16>(x, codes, scales, (int)N, (int)(K / kMxBlock), y, stream);
}

}  // namespace woq
