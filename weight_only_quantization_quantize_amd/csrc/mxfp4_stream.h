// What the products that stream microscaled weights past a few rows of
// activations share.  A wave takes units of 16 weight rows by one super-step of
// 512 K (16 blocks): four loads of 4 rows x 256 contiguous bytes each, turned
// through LDS of its own into the operands of four steps of
// v_mfma_scale_f32_16x16x128_f8f6f4.
//
// In LDS block c of row r lies at position c ^ r of the row's 16, so neither
// side meets a bank conflict.  At step s lane (r, q) (r = lane % 16, q =
// lane / 16) takes block 4 q + s of the super-step: its four scale bytes are one
// dword and the instruction's byte select picks the step's.
#pragma once

#include <type_traits>

#include "mxfp4_device.h"

namespace woq {

constexpr int kSuper = 16;                          // blocks per super-step
constexpr int kUnitBytes = 16 * 256;                // codes of a unit
constexpr int kUnitStage = kUnitBytes + 64 * 4;     // and a scale dword per lane

// One K step of one chunk of 16 rows of split activations.
struct MxActivations {
  i32x8_t p0, p1, p2;
  int s;
};

// Where a lane finds its row's activations: byte offsets from a fragment that
// the whole wave shares.
struct MxPlace {
  uint32_t lo, hi, scale;
};
// frag_step: fragments from the shared one to the row's; at: the lane's place in it.
__device__ inline MxPlace mx_place(int frag_step, int at) {
  return MxPlace{(uint32_t)(frag_step * kMxFragBytes + 16 * at), (uint32_t)(frag_step * kMxFragBytes + 1024 + 8 * at),
                 (uint32_t)(frag_step * kMxFragScaleBytes + 4 * at)};
}
__device__ inline void mx_load_activations(MxActivations& a, const uint8_t* __restrict__ frag,
                                           const uint8_t* __restrict__ fscale, const MxPlace& at) {
  auto piece = [&](int p) {
    return mx_operand(*reinterpret_cast<const u32x4_t*>(frag + p * kMxPieceBytes + at.lo),
                      *reinterpret_cast<const u32x2_t*>(frag + p * kMxPieceBytes + at.hi));
  };
  a.p0 = piece(0);
  a.p1 = piece(1);
  a.p2 = piece(2);
  a.s = *reinterpret_cast<const int*>(fscale + at.scale);
}

// A unit on its way: the codes of 16 rows and the lane's scale dword.
struct MxUnit {
  u32x4_t c[4];
  uint32_t s;
};

// rows: the unit's rows; codes, scales: their first; last: the last row that may
// be read (the others repeat it); scales_left: scale bytes from `scales` to the
// end of the array.  Blocks past the row's end repeat its last one: the
// activations are zeros there.
__device__ inline void mx_load_unit(MxUnit& u, const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                    int last, int64_t scales_left, int nblk, int S, int lane) {
  const int r = lane & 15, q = lane >> 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int lr = 4 * j + q, n = lr < last ? lr : last;
    int b = kSuper * S + (r ^ lr);
    b = b < nblk ? b : nblk - 1;
    u.c[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(codes + (uint32_t)(n * nblk + b) * 16u));
  }
  const uint32_t at = (uint32_t)((r < last ? r : last) * nblk + kSuper * S + 4 * q);
  const uint32_t end = scales_left - 4 < 0xFFFFFFFFll ? (uint32_t)(scales_left - 4) : 0xFFFFFFFFu;
  __builtin_memcpy(&u.s, scales + (at < end ? at : end), 4);
}

// The unit's codes and scales into the wave's LDS; scale bytes of blocks past
// the row's end become 127 (they may be another row's, and a NaN scale would
// survive the zeros).
__device__ inline void mx_stage_unit(const MxUnit& u, uint8_t* __restrict__ stage, int last, int64_t scales_left,
                                     int nblk, int S, int lane) {
  const int r = lane & 15, q = lane >> 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) *reinterpret_cast<u32x4_t*>(stage + 1024 * j + 16 * lane) = u.c[j];
  const uint32_t at = (uint32_t)((r < last ? r : last) * nblk + kSuper * S + 4 * q);
  const uint32_t end = scales_left - 4 < 0xFFFFFFFFll ? (uint32_t)(scales_left - 4) : 0xFFFFFFFFu;
  const int live = nblk - (kSuper * S + 4 * q);  // of the lane's four blocks
  const uint32_t mask = live >= 4 ? 0xFFFFFFFFu : (live <= 0 ? 0u : (1u << (8 * live)) - 1u);
  const uint32_t v = at <= end ? u.s : u.s >> (8 * ((at - end) & 3));
  *reinterpret_cast<uint32_t*>(stage + kUnitBytes + 4 * lane) = (v & mask) | (0x7F7F7F7Fu & ~mask);
}

__device__ inline i32x8_t mx_staged_weights(const uint8_t* __restrict__ stage, int s, int lane) {
  const int r = lane & 15, q = lane >> 4;
  return mx_operand(*reinterpret_cast<const u32x4_t*>(stage + 256 * r + 16 * ((4 * q + s) ^ r)));
}
__device__ inline int mx_staged_scale(const uint8_t* __restrict__ stage, int lane) {
  return *reinterpret_cast<const int*>(stage + kUnitBytes + 4 * lane);
}

// acc (rows: activations, columns: weights) += step S of a unit, smallest piece first.
template <int S>
__device__ inline void mx_multiply(float4_t& acc, const MxActivations& a, i32x8_t w, int scale) {
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.p2, w, acc, kMfmaFp6, kMfmaFp4, 2, a.s, S, scale);
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.p1, w, acc, kMfmaFp6, kMfmaFp4, 1, a.s, S, scale);
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.p0, w, acc, kMfmaFp6, kMfmaFp4, 0, a.s, S, scale);
}

// f(integral_constant s) for the four steps of a super-step.
template <class F>
__device__ inline void mx_each_step(F&& f) {
  f(std::integral_constant<int, 0>{});
  f(std::integral_constant<int, 1>{});
  f(std::integral_constant<int, 2>{});
  f(std::integral_constant<int, 3>{});
}

}  // namespace woq
