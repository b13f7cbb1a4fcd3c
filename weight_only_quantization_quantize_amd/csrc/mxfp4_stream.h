// What the products that stream microscaled weights past a few rows of
// activations share.  A wave takes units of 16 weight rows by one super-step of
// 512 K (16 blocks): four loads of 4 rows x 256 contiguous bytes each, turned
// through LDS of its own into the operands of four steps of 128 K: one
// v_mfma_scale_f32_16x16x128_f8f6f4 each with 4-bit activations, four
// v_mfma_f32_16x16x32 of widened weights with 16-bit ones.
//
// In LDS block c of row r lies at position c ^ r of the row's 16, so neither
// side meets a bank conflict.  At step s lane (r, q) (r = lane % 16, q =
// lane / 16) takes block 4 q + s of the super-step: its four scale bytes are one
// dword, of which a step takes one byte.
#pragma once

#include <type_traits>

#include "mxfp4_device.h"

namespace woq {

constexpr int kSuper = 16;                          // blocks per super-step
constexpr int kUnitBytes = 16 * 256;                // codes of a unit
constexpr int kUnitStage = kUnitBytes + 64 * 4;     // and a scale dword per lane

// A super-step of one chunk of 16 rows of 16-bit activations: a lane's blocks 4 q ..
// 4 q + 3 of it, one for each step.
typedef u32x4_t MxActivations[4][4];

// row: the lane's row of X [., 32 nblk].  Blocks past its end are read as its last
// one; mx_mask_activations clears them, at a place of its own because a first use
// waits for the loads.
__device__ __forceinline__ void mx_load_activations(MxActivations& x, const uint16_t* __restrict__ row, int nblk, int S, int lane) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int b = kSuper * S + 4 * (lane >> 4) + s;
    const u32x4_t* const p = reinterpret_cast<const u32x4_t*>(row + (uint32_t)((b < nblk ? b : nblk - 1) * kMxBlock));
#pragma unroll
    for (int j = 0; j < 4; ++j) x[s][j] = p[j];
  }
}
__device__ __forceinline__ void mx_mask_activations(MxActivations& x, int nblk, int S, int lane) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const bool live = kSuper * S + 4 * (lane >> 4) + s < nblk;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[s][j][e] = live ? x[s][j][e] : 0u;
  }
}
// frag: the super-step's four fragments; at: the lane's place in them (16 times the
// lane for its own row).
__device__ __forceinline__ void mx_load_fragments(MxActivations& x, const uint8_t* __restrict__ frag, uint32_t at) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) x[s][j] = *reinterpret_cast<const u32x4_t*>(frag + s * kMxFragBytes + 1024 * j + at);
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
  const uint32_t end = (scales_left - 4) >> 32 ? 0xFFFFFFFFu : (uint32_t)(scales_left - 4);
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
  const uint32_t end = (scales_left - 4) >> 32 ? 0xFFFFFFFFu : (uint32_t)(scales_left - 4);
  const int live = nblk - (kSuper * S + 4 * q);  // of the lane's four blocks
  const uint32_t mask = live >= 4 ? 0xFFFFFFFFu : (live <= 0 ? 0u : (1u << (8 * live)) - 1u);
  const uint32_t v = at <= end ? u.s : u.s >> (8 * ((at - end) & 3));
  *reinterpret_cast<uint32_t*>(stage + kUnitBytes + 4 * lane) = (v & mask) | (0x7F7F7F7Fu & ~mask);
}

__device__ inline u32x4_t mx_staged_weights(const uint8_t* __restrict__ stage, int s, int lane) {
  const int r = lane & 15, q = lane >> 4;
  return *reinterpret_cast<const u32x4_t*>(stage + 256 * r + 16 * ((4 * q + s) ^ r));
}
__device__ inline uint32_t mx_staged_scale(const uint8_t* __restrict__ stage, int lane) {
  return *reinterpret_cast<const uint32_t*>(stage + kUnitBytes + 4 * lane);
}

// f(integral_constant s) for the four steps of a super-step.
template <class F>
__device__ inline void mx_each_step(F&& f) {
  f(std::integral_constant<int, 0>{});
  f(std::integral_constant<int, 1>{});
  f(std::integral_constant<int, 2>{});
  f(std::integral_constant<int, 3>{});
}

// acc (rows: activations, columns: weights) += the staged unit's product over kMxGain
// with its super-step of 16-bit activations x, and also += that with more, where TWO is
// set.  The usual way is straight code of its own, so that conversions run beside the
// matrix instructions.
template <class XT, bool TWO>
__device__ __forceinline__ void mx_multiply_unit(float4_t& acc, const MxActivations& x, float4_t& also, const MxActivations& more,
                                                 const uint8_t* __restrict__ stage, int lane) {
  const uint32_t scale = mx_staged_scale(stage, lane);
  auto step = [&](auto sel, auto widen) {
    constexpr int s = decltype(sel)::value;
    const u32x4_t c = mx_staged_weights(stage, s, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x4_t w = widen(c[j], scale >> (8 * s) & 0xFFu);
      if constexpr (TWO) also = XT::mfma16x16x32(more[s][j], w, also);
      acc = XT::mfma16x16x32(x[s][j], w, acc);
    }
  };
  auto usual = [](uint32_t c, uint32_t b) { return mx_widen<XT>(c, b); };
  if (!__any(mx_unusual<XT>(scale, 4))) {
    mx_each_step([&](auto sel) { step(sel, usual); });
    return;
  }
  mx_each_step([&](auto sel) {
    constexpr int s = decltype(sel)::value;
    const uint32_t b = scale >> (8 * s) & 0xFFu;
    const u32x4_t c = mx_staged_weights(stage, s, lane);
    if (!__any(mx_needs_care<XT>(c, b))) {
      step(sel, usual);
    } else if constexpr (!kMxIsF16<XT>) {
      step(sel, [](uint32_t c, uint32_t b) { return mx_widen_any(c, b); });
    } else {
      const bool large = __any(mx_large(b));
#pragma unroll 1
      for (int p = 0; p < kMxPasses; p += large ? 1 : 4)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc = BF16::mfma16x16x32(mx_general_activations(x[s][j], p), mx_general_weights(c[j], b, p), acc);
    }
  });
}
template <class XT>
__device__ __forceinline__ void mx_multiply_unit(float4_t& acc, const MxActivations& x, const uint8_t* __restrict__ stage, int lane) {
  float4_t none;
  mx_multiply_unit<XT, false>(acc, x, none, x, stage, lane);
}

}  // namespace woq
