// Matrix products with a microscaled 4-bit right operand W [N, K]:
//   Mx         a microscaled 4-bit left operand A [M, K], both as stored, inside
//              v_mfma_scale_f32_32x32x64_f8f6f4: no element is decoded;
//   F16, BF16  16-bit activations, by weights widened to their type in registers on
//              v_mfma_f32_32x32x16 (mxfp4_device.h).
// Y[m, n] = sum over the 32-element blocks b of 2^(sA + sW - 254) sum_k a w: the
// products are exact and the sums are the matrix unit's fp32.
//
// Tile.  A group of 2 x WN waves computes 64 TM x 32 WN TN of Y, a wave 32 TM x
// 32 TN; KG groups of a workgroup share a tile's K and add their sums through
// LDS at the end.  `launch` chooses: where there is work for all compute units
// the matrix instructions bound the product and the largest tile wins (16-bit A is
// the heavier operand, 2 bytes an element against 17 / 32, and gets the shorter side;
// two workgroups of that tile share a compute unit, which hides the one's barriers,
// prologue and stores behind the other's instructions).
// Below that the number of stages in flight counts: small tiles, K split.
// 2048 x 11008 x 4096 takes 165 .. 172 us with 16-bit activations (1.1 P flop/s; a
// library product of 16-bit matrices reaches 1.16 P) and 57 us with 4-bit ones (3.2 P of
// the 6.7 P that the matrix unit reaches on registers alone).  For 4-bit operands the vector instructions beside the matrix ones count (LDS is busy
// for 28% of the time): masks of the last blocks, a shift for every scale and addresses
// from their parts, 90 instructions for 16 matrix instructions in place of 20, took 63.
//
// Pipeline.  K goes in stages of 64 KS, kStages of them in LDS, filled by direct
// loads (global_load_lds: no registers, no instructions to write LDS).  At the top
// of a turn a wave waits until its own loads of this stage are done, meets the
// others at the barrier, which also says that everybody is through with the
// previous stage, starts the loads of the stage kStages - 1 ahead into that one's
// place, and multiplies.  The loads are written out in assembly because the
// compiler would wait for all of them before every read of LDS; their counter is
// waited for by hand, and there is no other vector memory access inside the loop.
// Longer stages mean fewer barriers: 256 of K for 4-bit operands and K split
// between two groups of waves took 333 x 1001 x 5152 from 15 to 10 us; the large
// tile of 16-bit ones keeps 64, which leave it two workgroups a compute unit (2048 x
// 11008 x 4096: 177 us with the pass before it, 188 with 128; 184 with 256 x 128 tiles).
//
// Scales.  The 4-bit operands' scale bytes lie K / 32 bytes apart from row to row
// at any alignment, which direct loads cannot gather; turn_scales
// (mxfp4_quantize.hip; 16-bit activations: in the launch that lays these out) makes
// them one dword per row and 128 of K, rows contiguous.  Small tiles of two 4-bit operands do
// that themselves, into LDS, once for all of K.  Past a row's end stands its last
// block again, with scale byte 0: the product of two such blocks is below fp32's
// smallest number (and 16-bit activations are zeros there), so no operand is masked.
//
// LDS layout of a 4-bit operand: a row's 32 KS bytes of a stage are chunks of
// one block each, chunk c at position c ^ swizzle(row), so that 16 rows read at
// one chunk lie in 16 different 16-byte slots of the 256-byte bank row.
//
// Tile order.  Workgroup b runs on XCD b % 8; each XCD takes one contiguous run of
// tiles, in groups of 8 M tiles, M fastest, so that the tiles in flight there (32 or
// 64) share about as much of A as of W in its L2.  All M tiles in one group take 67 us
// in place of 64 .. 66 for 2048 x 11008 x 4096 of 4-bit operands, and the same 177 with
// 16-bit activations.
#include <type_traits>

#include "mxfp4_device.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kXcds = 8;
constexpr int kGroup = 8;  // M tiles of a group

typedef __attribute__((address_space(3))) uint8_t lds_byte;

__device__ inline uint32_t lds_address(const void* p) { return (uint32_t)(uintptr_t)(const lds_byte*)p; }

// Direct loads to LDS: lane l's 16 (4) bytes from base + offset go to to + 16 l
// (4 l).  M0 holds the LDS address.  The five wait states cover the write of M0
// and a base address that a vector instruction wrote just before.  The caller
// waits for the data with wait_loads.  (The compiler reserves M0 and warns of it on a
// clobber list; it heeds the clobber where it sets M0 for itself.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ inline void load_lds16(const uint8_t* base, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base)
               : "m0", "memory");
}
__device__ inline void load_lds4(const uint8_t* base, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, %2" ::"s"(to), "v"(offset), "s"(base)
               : "m0", "memory");
}
#pragma clang diagnostic pop
// Until at most N of the wave's vector memory loads are under way and its LDS
// reads are done.
template <int N>
__device__ inline void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// A 4-bit operand: ROWS rows, stages of 64 KS (KS 1, 2 or 4).  One load of a wave
// takes 32 / KS rows.
template <int ROWS, int KS>
struct Tile4 {
  static constexpr int kRowBytes = 32 * KS;
  static constexpr int kBytes = ROWS * kRowBytes;
  static constexpr int kUnits = kBytes / 1024;
  static constexpr int kDwords = KS == 4 ? 2 : 1;  // scale dwords of a row's stage, [dword][row]
  static constexpr int kScaleUnits = ROWS / 64 * kDwords;
  static constexpr int kScaleBytes = ROWS * 4 * kDwords;
  static_assert(kMxScaleRowPad % ROWS == 0, "a tile's scale loads stay inside the padded array");
  const uint8_t* codes;
  const uint8_t* scales;
  uint32_t scale_step;  // bytes between K tiles of the scale dwords
  int nblk, last, chunk;

  __device__ static int swizzle(int row) { return KS == 4 ? (row >> 1) & 7 : (KS == 2 ? (row >> 2) & 3 : (row >> 3) & 1); }
  __device__ void start(const uint8_t* codes_, const uint8_t* scales_, int row0, int rows, int rows_pad, int nblk_, int) {
    nblk = nblk_;
    codes = codes_ + (int64_t)row0 * nblk * 16;
    scales = scales_ + (int64_t)row0 * 4;
    scale_step = (uint32_t)rows_pad * 4u;
    last = rows - row0 - 1;
    const int lane = threadIdx.x & 63;
    chunk = (lane & (2 * KS - 1)) ^ swizzle(lane / (2 * KS));
  }
  __device__ void load(int unit, int h, uint32_t to) const {
    const int lane = threadIdx.x & 63;
    int r = unit * (32 / KS) + lane / (2 * KS);
    r = r < last ? r : last;
    // (KS = 4: a load's 8 rows take every other half of the swizzle)
    int b = 2 * KS * h + (KS == 4 ? chunk ^ ((unit & 1) << 2) : chunk);
    b = b < nblk ? b : nblk - 1;  // past the row's end: its last block, at scale 2^-127
    load_lds16(codes, (uint32_t)(r * nblk + b) * 16u, to + 1024u * (uint32_t)unit);
  }
  __device__ void load_scales(int unit, int h, uint32_t to) const {
    const int kt = KS == 1 ? h >> 1 : kDwords * h + unit / (ROWS / 64);
    const uint32_t rows = 256u * (uint32_t)(unit % (ROWS / 64));
    load_lds4(scales + (int64_t)kt * scale_step, rows + 4u * (threadIdx.x & 63), to + 256u * (uint32_t)unit);
  }
  // lane (row, half) multiplies block 2 s + half of its row's stage; 32 rows on, 32
  // kRowBytes on
  __device__ static uint32_t place(int row, int s, int half) {
    return (uint32_t)(row * kRowBytes + ((2 * s + half) ^ swizzle(row)) * 16);
  }
  // Step s's scale.  A row's dword holds blocks 0, 2, 1, 3 of its 128 K: the lane
  // reads its half's two (at: 2 half into the row's place), and the instruction's
  // byte select, the same for all lanes, picks the step; one byte where a stage has
  // one step.
  __device__ static int scale(const uint8_t* at, int s, int h) {
    if constexpr (KS == 1) return (int)at[h & 1];
    return (int)*reinterpret_cast<const uint16_t*>(at + 4 * ROWS * (KS == 4 ? s >> 1 : 0));
  }
  static constexpr int select(int s) { return KS == 1 ? 0 : s & 1; }
};

// 16-bit activations: stages of KS fragments (64 of K each) of each 32 rows.
template <int ROWS, int KS>
struct TileRows {
  static constexpr int kBytes = ROWS / 32 * KS * kMxFragBytes;
  static constexpr int kUnits = kBytes / 1024;
  static constexpr int kScaleUnits = 0, kScaleBytes = 0;
  const uint8_t* frags;
  uint32_t ksteps;

  __device__ void start(const uint8_t* frags_, const uint8_t*, int row0, int, int, int, int ksteps_) {
    ksteps = (uint32_t)ksteps_;
    frags = frags_ + (int64_t)(row0 / 32) * ksteps * kMxFragBytes;
  }
  __device__ void load(int unit, int h, uint32_t to) const {
    constexpr uint32_t kUnitsOf = KS * kMxFragBytes / 1024;  // of 32 rows
    const uint32_t rg = (uint32_t)unit / kUnitsOf, in = (uint32_t)unit % kUnitsOf;
    load_lds16(frags + (int64_t)h * KS * kMxFragBytes, rg * ksteps * kMxFragBytes + 1024u * in + 16u * (threadIdx.x & 63),
               to + 1024u * (uint32_t)unit);
  }
  __device__ void load_scales(int, int, uint32_t) const {}
};

// RES > 0: the tile's scale bytes for all of K (at most 128 RES) stay in LDS, a dword
// for a row and 128 of K.
constexpr int kResident = 28, kResidentAlone = 128;
// XT: the activations' 16-bit type, or Mx.
struct Mx {};
template <class XT, int TM, int TN, int WN, int KS, int KG, int RES>
struct Config {
  static constexpr int kWaves = 2 * WN, kThreads = 64 * kWaves * KG;
  static constexpr bool kRows = !std::is_same_v<XT, Mx>;
  static constexpr int kKS = KS;
  static constexpr int BM = 64 * TM, BN = 32 * WN * TN;
  using TA = std::conditional_t<kRows, TileRows<BM, KS>, Tile4<BM, KS>>;
  using TW = Tile4<BN, kKS>;
  static constexpr int kStage = TA::kBytes + TW::kBytes + (RES ? 0 : TA::kScaleBytes + TW::kScaleBytes);
  // as many stages as leave room for a second workgroup, or, where that would be
  // fewer than two or there is none (kResidentAlone), as fill the LDS; at most 4
  static constexpr int kRoom = RES >= kResidentAlone ? 160 * 1024 - RES * 4 * (BM + BN) : (KG * kStage * 2 > 80 * 1024 ? 160 : 80) * 1024;
  static constexpr int kFit = kRoom / (KG * kStage);
  static constexpr int kStages = kFit > 4 ? 4 : (kFit < 2 ? 2 : kFit);
  static constexpr int per_wave(int units) { return (units + kWaves - 1) / kWaves; }
  static constexpr int kALoads = per_wave(TA::kUnits), kWLoads = per_wave(TW::kUnits);
  static constexpr int kAScaleLoads = RES ? 0 : per_wave(TA::kScaleUnits), kWScaleLoads = RES ? 0 : per_wave(TW::kScaleUnits);
  static constexpr int kLoads = kALoads + kWLoads + kAScaleLoads + kWScaleLoads;
};

template <class YT, class XT, int TM, int TN, int WN, int KS, int KG, int RES>
__global__ __launch_bounds__((Config<XT, TM, TN, WN, KS, KG, RES>::kThreads), 2) void mxfp4_gemm_kernel(const uint8_t* __restrict__ A,
                                                                 const uint8_t* __restrict__ As,
                                                                 const uint8_t* __restrict__ W,
                                                                 const uint8_t* __restrict__ Ws, int M, int N,
                                                                 int m_pad, int n_pad, int nblk, int mtiles, int tiles,
                                                                 uint16_t* __restrict__ Y) {
  using C = Config<XT, TM, TN, WN, KS, KG, RES>;
  constexpr int kWaves = C::kWaves;
  using TA = typename C::TA;
  using TW = typename C::TW;
  constexpr int kAt = TA::kBytes, kAsAt = kAt + TW::kBytes, kWsAt = kAsAt + TA::kScaleBytes;
  __shared__ __attribute__((aligned(1024))) uint8_t lds_all[KG][C::kStages][C::kStage];
  __shared__ uint32_t a_scales[RES ? RES : 1][RES ? C::BM : 1], w_scales[RES ? RES : 1][RES ? C::BN : 1];

  const int per = (tiles + kXcds - 1) / kXcds;
  const int tile = (int)(blockIdx.x % kXcds) * per + (int)(blockIdx.x / kXcds);
  if (tile >= tiles) return;
  const int gtiles = kGroup * (tiles / mtiles);  // of a group of M tiles
  const int g = tile / gtiles, gm = mtiles - g * kGroup < kGroup ? mtiles - g * kGroup : kGroup;
  const int m0 = (g * kGroup + tile % gtiles % gm) * C::BM, n0 = tile % gtiles / gm * C::BN;
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = wave_all % kWaves, group = wave_all / kWaves;
  const int wm = (wave & 1) * TM, wn = (wave >> 1) * TN;  // in units of 32 rows
  const int half = lane >> 5, r32 = lane & 31;
  // K group `group` takes the stages [h0, h1); all groups make the same number of turns
  const int stages = (nblk + 2 * C::kKS - 1) / (2 * C::kKS);
  const int turns = (stages + KG - 1) / KG;
  const int h0 = group * turns, h1 = h0 + turns < stages ? h0 + turns : stages;
  uint8_t(*const lds)[C::kStage] = lds_all[group];

  TA ta;
  TW tw;
  ta.start(A, As, m0, M, m_pad, nblk, ((nblk + 3) >> 2) * 2);
  tw.start(W, Ws, n0, N, n_pad, nblk, 0);
  // every wave starts the same number of loads a stage: past an operand's units
  // the last one is loaded again, past the last stage that stage
  auto issue = [&](int h_, int buf) {
    const int h = h_ < stages ? h_ : stages - 1;
    const uint32_t to = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_address(lds[0])) + (uint32_t)(buf * C::kStage);
    auto unit = [&](int j, int units) {
      const int u = wave + kWaves * j;
      return u < units ? u : units - 1;
    };
#pragma unroll
    for (int j = 0; j < C::kALoads; ++j) ta.load(unit(j, TA::kUnits), h, to);
#pragma unroll
    for (int j = 0; j < C::kWLoads; ++j) tw.load(unit(j, TW::kUnits), h, to + kAt);
#pragma unroll
    for (int j = 0; j < C::kAScaleLoads; ++j) ta.load_scales(unit(j, TA::kScaleUnits), h, to + kAsAt);
#pragma unroll
    for (int j = 0; j < C::kWScaleLoads; ++j) tw.load_scales(unit(j, TW::kScaleUnits), h, to + kWsAt);
  };

  // where the lane's operands lie in a stage: computed once, so that a stage costs one
  // addition for each step
  uint32_t a_at[KS], w_at[KS], as_at = 0, ws_at = kWsAt + 4 * (wn * 32 + r32) + 2 * half;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    w_at[s] = kAt + TW::place((wn * 32) + r32, s, half);
    a_at[s] = 0;
    if constexpr (!C::kRows) a_at[s] = TA::place(wm * 32 + r32, s, half);
    asm volatile("" : "+v"(w_at[s]), "+v"(a_at[s]));
  }
  if constexpr (!C::kRows) as_at = kAsAt + 4 * (wm * 32 + r32) + 2 * half;
  const uint32_t a_at0 = (uint32_t)(wm * KS * kMxFragBytes + 16 * lane);
  asm volatile("" : "+v"(as_at), "+v"(ws_at));

  float16_t acc[TM][TN];
  // All of K.  16-bit activations: in the usual way (part 0), or (part 1, and 2 for the
  // second half of the columns of a tile whose sums fill the registers) each step in the
  // way it needs; returns whether the lane met a block that the usual one does not
  // multiply.  Both ways in one loop spill or hold up the usual one.  A block of scale
  // byte 100 in every 256 rows, fp16: 2048 x 11008 x 4096 190 -> 430 us, 64 x 11008 x 4096
  // 19 -> 34 (every step of such a tile in the general way: 890 and 109).
  constexpr int kParts = TM * TN > 4 ? 2 : 1;
  auto all_of_k = [&](auto part) {
    constexpr bool kGeneral = decltype(part)::value > 0;
    constexpr int kFrom = kGeneral ? (decltype(part)::value - 1) * (TN / kParts) : 0, kTo = kGeneral ? kFrom + TN / kParts : TN;
    bool general = false;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = kFrom; j < kTo; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    for (int st = 0; st + 1 < C::kStages; ++st) issue(h0 + st, st);
    if constexpr (RES > 0) {  // seen by all behind the first turn's barrier
      static_assert(KS == 4 && !C::kRows && RES % 4 == 0);
      const int chunks = (nblk + 15) >> 4;
      for (int i = threadIdx.x; i < (C::BM + C::BN) * chunks; i += C::kThreads) {
        const int row = i % (C::BM + C::BN), g = i / (C::BM + C::BN);
        const bool of_a = row < C::BM;
        const int r = of_a ? m0 + row : n0 + row - C::BM, last = (of_a ? M : N) - 1;
        const u32x4_t v = mx_scale_chunk((of_a ? As : Ws) + (int64_t)(r < last ? r : last) * nblk, g, nblk, 0u);
        uint32_t* const to = of_a ? &a_scales[4 * g][row] : &w_scales[4 * g][row - C::BM];
#pragma unroll
        for (int q = 0; q < 4; ++q) to[q * (of_a ? C::BM : C::BN)] = v[q];
      }
    }
    int buf = 0;
    for (int h = h0; h < h0 + turns; ++h) {
      wait_loads<(C::kStages - 2) * C::kLoads>();
      __builtin_amdgcn_s_barrier();
      issue(h + C::kStages - 1, buf == 0 ? C::kStages - 1 : buf - 1);
      const uint8_t* const la = lds[buf];
      buf = buf + 1 == C::kStages ? 0 : buf + 1;
      if (KG > 1 && h >= h1) continue;
      auto multiply = [&](auto sel) {
        constexpr int s = decltype(sel)::value;
        u32x4_t wc[TN];
        int bs[TN];
#pragma unroll
        for (int j = kFrom; j < kTo; ++j) {
          wc[j] = *reinterpret_cast<const u32x4_t*>(la + w_at[s] + j * 32 * TW::kRowBytes);
          if constexpr (RES > 0)
            bs[j] = (int)reinterpret_cast<const uint16_t*>(&w_scales[2 * h + (s >> 1)][(wn + j) * 32 + r32])[half];
          else
            bs[j] = TW::scale(la + ws_at + 128 * j, s, h);
        }
        if constexpr (!C::kRows) {
#pragma unroll
          for (int i = 0; i < TM; ++i) {
            const i32x8_t v = mx_operand(*reinterpret_cast<const u32x4_t*>(la + a_at[s] + i * 32 * TA::kRowBytes));
            int as;
            if constexpr (RES > 0)
              as = (int)reinterpret_cast<const uint16_t*>(&a_scales[2 * h + (s >> 1)][(wm + i) * 32 + r32])[half];
            else
              as = TA::scale(la + as_at + 128 * i, s, h);
#pragma unroll
            for (int j = kFrom; j < kTo; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(wc[j]), v, acc[i][j], kMfmaFp4, kMfmaFp4,
                                                                          TW::select(s), bs[j], TA::select(s), as);
          }
        } else {
          auto acts = [&](int i, int q) {
            return *reinterpret_cast<const u32x4_t*>(la + a_at0 + ((i * KS + s) * 4 + q) * 1024);
          };
#pragma unroll
          for (int j = kFrom; j < kTo; ++j) bs[j] = bs[j] >> (8 * TW::select(s)) & 0xFF;
          auto step = [&](auto widen) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              u32x4_t w[TN];
#pragma unroll
              for (int j = kFrom; j < kTo; ++j) w[j] = widen(wc[j][q], (uint32_t)bs[j]);
#pragma unroll
              for (int i = 0; i < TM; ++i) {
                const u32x4_t x = acts(i, q);
#pragma unroll
                for (int j = kFrom; j < kTo; ++j) acc[i][j] = mfma32x32x16<XT>(w[j], x, acc[i][j]);
              }
            }
          };
          if constexpr (!kGeneral) {
            bool unusual = false;
#pragma unroll
            for (int j = kFrom; j < kTo; ++j) unusual |= mx_unusual<XT>((uint32_t)bs[j], 1);
            if (__any(unusual))
#pragma unroll
              for (int j = kFrom; j < kTo; ++j) general |= mx_needs_care<XT>(wc[j], (uint32_t)bs[j]);
            step([](uint32_t c, uint32_t b) { return mx_widen<XT>(c, b); });
          } else {
            bool care = false;
#pragma unroll
            for (int j = kFrom; j < kTo; ++j) care |= mx_needs_care<XT>(wc[j], (uint32_t)bs[j]);
            if (!__any(care)) {
              step([](uint32_t c, uint32_t b) { return mx_widen<XT>(c, b); });
            } else if constexpr (!kMxIsF16<XT>) {
              step([](uint32_t c, uint32_t b) { return mx_widen_any(c, b); });
            } else {
              bool large = false;
#pragma unroll
              for (int j = kFrom; j < kTo; ++j) large |= mx_large((uint32_t)bs[j]);
              large = __any(large);
#pragma unroll 1
              for (int p = 0; p < kMxPasses; p += large ? 1 : 4)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  asm volatile("" ::: "memory");  // activations are read again each pass: kept, they spill
                  u32x4_t w[TN];
#pragma unroll
                  for (int j = kFrom; j < kTo; ++j) w[j] = mx_general_weights(wc[j][q], (uint32_t)bs[j], p);
#pragma unroll
                  for (int i = 0; i < TM; ++i) {
                    const u32x4_t x = mx_general_activations(acts(i, q), p);
#pragma unroll
                    for (int j = kFrom; j < kTo; ++j) acc[i][j] = mfma32x32x16<BF16>(w[j], x, acc[i][j]);
                  }
                }
            }
          }
        }
      };
      multiply(std::integral_constant<int, 0>{});
      if constexpr (KS > 1) multiply(std::integral_constant<int, 1>{});
      if constexpr (KS > 2) {
        multiply(std::integral_constant<int, 2>{});
        multiply(std::integral_constant<int, 3>{});
      }
    }
    wait_loads<0>();  // none may land in LDS that is another workgroup's by then
    return general;
  };
  if constexpr (C::kRows) {
    __shared__ bool any_general;
    if (threadIdx.x == 0) any_general = false;  // before the first turn's barrier
    if (all_of_k(std::integral_constant<int, 0>{})) any_general = true;
    __syncthreads();
    if (any_general) {  // the tile again, for all of its waves
      all_of_k(std::integral_constant<int, 1>{});
      if constexpr (kParts == 2) {
        __syncthreads();
        all_of_k(std::integral_constant<int, 2>{});
      }
    }
  } else {
    all_of_k(std::integral_constant<int, 0>{});
  }
  __syncthreads();  // nobody reads operands any more

  if constexpr (KG > 1) {
    // the groups' sums meet in LDS, [wave][tile][lane], added in order
    static_assert(TM * TN * kWaves * 4096 <= C::kStages * C::kStage, "a group's sums fit its stages' place");
    float16_t* const mine = reinterpret_cast<float16_t*>(&lds[0][0]) + wave * TM * TN * 64 + lane;
    if (group)
#pragma unroll
      for (int i = 0; i < TM * TN; ++i) mine[i * 64] = acc[i / TN][i % TN];
    __syncthreads();
    if (group) return;
#pragma unroll
    for (int g = 1; g < KG; ++g) {
      const float16_t* const other = reinterpret_cast<const float16_t*>(&lds_all[g][0][0]) + wave * TM * TN * 64 + lane;
#pragma unroll
      for (int i = 0; i < TM * TN; ++i) {
        const float16_t v = other[i * 64];
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i / TN][i % TN][e] += v[e];
      }
    }
  }

  // D: lane holds row r32 of Y and columns 8 (e / 4) + 4 half + e % 4 (W is the
  // instruction's first operand for that).  Each wave turns 32 rows at a time
  // through LDS of its own, so that Y is written in whole rows of the wave's
  // columns, 16 bytes a lane.
  constexpr float kGain = [] {
    if constexpr (C::kRows) return kMxGain<XT>;
    return 1.0f;
  }();
  constexpr int kPitch = 64 * TN + 16, kChunks = 4 * TN;
  static_assert(kWaves * 32 * kPitch <= C::kStages * C::kStage, "the turn fits the stages' place");
  uint8_t* const turn = &lds[0][0] + wave * 32 * kPitch;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t lo = (uint32_t)YT::from_f32(acc[i][j][4 * g] * kGain) | (uint32_t)YT::from_f32(acc[i][j][4 * g + 1] * kGain) << 16;
        const uint32_t hi = (uint32_t)YT::from_f32(acc[i][j][4 * g + 2] * kGain) | (uint32_t)YT::from_f32(acc[i][j][4 * g + 3] * kGain) << 16;
        *reinterpret_cast<u32x2_t*>(turn + r32 * kPitch + 64 * j + 16 * g + 8 * half) = u32x2_t{lo, hi};
      }
    asm volatile("" ::: "memory");
#pragma unroll
    for (int q = 0; q < 32 * kChunks / 64; ++q) {
      const int row = (64 * q + lane) / kChunks, ch = (64 * q + lane) % kChunks;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(turn + row * kPitch + 16 * ch);
      const int m = m0 + (wm + i) * 32 + row, n = n0 + wn * 32 + 8 * ch;
      if (m < M && n < N) {
        uint16_t* const y = Y + (int64_t)m * N + n;
        if (n + 8 <= N) {
          __builtin_memcpy(y, &v, 16);  // of any alignment: N may be odd
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < N) y[e] = (uint16_t)(v[e / 2] >> (16 * (e % 2)));
        }
      }
    }
    asm volatile("" ::: "memory");
  }
}

size_t scale_bytes(int64_t rows, int64_t K) { return (size_t)mxfp4_scale_rows(rows) * (size_t)((K + 255) / 256 * 2) * 4; }

template <class YT, class XT, int TM, int TN, int WN, int KS, int KG, int RES = 0>
hipError_t launch_tiles(const void* A, const void* As, const void* W, const void* Ws, int64_t M, int64_t N, int64_t K,
                        void* Y, hipStream_t stream) {
  using C = Config<XT, TM, TN, WN, KS, KG, RES>;
  const int64_t mt = (M + C::BM - 1) / C::BM, nt = (N + C::BN - 1) / C::BN;
  const int64_t tiles = mt * nt;
  const unsigned grid = (unsigned)((tiles + kXcds - 1) / kXcds * kXcds);
  mxfp4_gemm_kernel<YT, XT, TM, TN, WN, KS, KG, RES><<<grid, C::kThreads, 0, stream>>>(
      static_cast<const uint8_t*>(A), static_cast<const uint8_t*>(As), static_cast<const uint8_t*>(W),
      static_cast<const uint8_t*>(Ws), (int)M, (int)N, (int)mxfp4_scale_rows(M), (int)mxfp4_scale_rows(N), (int)(K / kMxBlock), (int)mt,
      (int)tiles, static_cast<uint16_t*>(Y));
  return hipGetLastError();
}

// The tile with the smallest time by a model of what was measured at K = 4096, in us
// for n = ceil(tiles / 256) tiles a compute unit (16-bit: with the pass before it):
//   4-bit A:   256 x 256 36 n          (2048 x 8192: 41;  1024 x 28672, K / 2: 49)
//              128 x 128 6 + 10 n      (n = 1: 15 .. 21, 2: 23 .. 25, 4: 46, 6: 63 .. 65)
//              64 x 64   3 + 4.5 n     (n = 1: 8, 2: 11, 4: 22, 8: 34 .. 40)
//   16-bit A:  128 x 256 16 + 54 n     (n = 1: 59 .. 76, 2: 125, 3: 182)
//              64 x 256  8 + 30.5 n    (n = 1: 34 .. 45, 2: 73, 4: 136, 6: 190)
//              64 x 128  5 + 21.5 n    (n = 1: 23 .. 29, 2: 50, 4: 91, 8: 173)
//              64 x 64   6 + 14.5 n    (n = 1: 18 .. 22, 2: 37, 4: 66, 8: 122)
// Not all of it grows with K, but the order stays: at K = 32 .. 1024 and seven sizes
// from 16 x 4096 to 2048 x 8192 the choice is within 0.6 us of the best tile, 16-bit
// 64 x 28672 x 32 for one 7.3 us, with 64 x 256 6.8; 2048 x 8192 x 256 18.7, the others
// 19.0, 36 and 50; microscaled 1024 x 4096 x 256 7.3, the others 9.2 and 9.9.
// The small ones split K between two groups of waves.
int64_t per_cu(int64_t M, int64_t N, int bm, int bn) { return ((M + bm - 1) / bm * ((N + bn - 1) / bn) + 255) / 256; }
enum class Tile { kLarge, kMiddle, kSmall };
Tile tile_mx(int64_t M, int64_t N) {
  const double large = 36.0 * per_cu(M, N, 256, 256), mid = 6.0 + 10.0 * per_cu(M, N, 128, 128),
               small = 3.0 + 4.5 * per_cu(M, N, 64, 64);
  return large <= mid && large <= small ? Tile::kLarge : (mid <= small ? Tile::kMiddle : Tile::kSmall);
}
// Small 4-bit tiles keep the scales in LDS where that leaves a second workgroup a
// compute unit, or none is needed: no pass over them, no workspace.  Whole products
// with weights out of HBM, with / without: 333 x 1001 x 5152 10.3 / 12.9 us, 128 x 4096
// x 4096 8.0 / 10.7, 512 x 1024 x 1024 4.1 / 6.5, 256 x 8192 x 3584 11.7 / 14.3, 64 x 8192
// x 8192 15.4 / 21.4.  Those alone on their compute unit have three stages (with two:
// 64 x 8192 x 8192 18.9 us, 333 x 1001 x 5152 11.0).
bool resident(int64_t M, int64_t N, int64_t K) {
  return tile_mx(M, N) == Tile::kSmall && (K <= 128 * kResident || (K <= 128 * kResidentAlone && per_cu(M, N, 64, 64) == 1));
}

template <class YT, class XT>
hipError_t launch(const void* A, const void* As, const void* W, const void* Ws, int64_t M, int64_t N, int64_t K,
                  void* Y, hipStream_t stream) {
  if constexpr (std::is_same_v<XT, Mx>) {
    if (resident(M, N, K))
      return K <= 128 * kResident ? launch_tiles<YT, XT, 1, 1, 2, 4, 2, kResident>(A, As, W, Ws, M, N, K, Y, stream)
                                  : launch_tiles<YT, XT, 1, 1, 2, 4, 2, kResidentAlone>(A, As, W, Ws, M, N, K, Y, stream);
    switch (tile_mx(M, N)) {
      case Tile::kLarge: return launch_tiles<YT, XT, 4, 2, 4, 4, 1>(A, As, W, Ws, M, N, K, Y, stream);
      case Tile::kMiddle: return launch_tiles<YT, XT, 2, 2, 2, 4, 1>(A, As, W, Ws, M, N, K, Y, stream);
      default: return launch_tiles<YT, XT, 1, 1, 2, 4, 2>(A, As, W, Ws, M, N, K, Y, stream);
    }
  } else {
    const double large = 16.0 + 54.0 * per_cu(M, N, 128, 256), wide = 8.0 + 30.5 * per_cu(M, N, 64, 256),
                 mid = 5.0 + 21.5 * per_cu(M, N, 64, 128), small = 6.0 + 14.5 * per_cu(M, N, 64, 64);
    if (large <= wide && large <= mid && large <= small)
      return launch_tiles<YT, XT, 2, 4, 2, 1, 1>(A, As, W, Ws, M, N, K, Y, stream);
    if (wide <= mid && wide <= small) return launch_tiles<YT, XT, 1, 2, 4, 2, 1>(A, As, W, Ws, M, N, K, Y, stream);
    if (mid <= small) return launch_tiles<YT, XT, 1, 2, 2, 2, 2>(A, As, W, Ws, M, N, K, Y, stream);
    return launch_tiles<YT, XT, 1, 1, 2, 2, 2>(A, As, W, Ws, M, N, K, Y, stream);
  }
}

// Few rows, or small outputs, go to the weight-streaming kernels (K >= 128), which
// need no pass over the scales and cut no tile that is mostly empty.  Whole
// products, us, streaming / the best tile:
//   16-bit, 32 rows  8192 x 8192 22 / 33, 4096 x 11008 21 / 40, 28672 x 8192 43 .. 50 / 49,
//                    4096 x 4096 9 / 19, 16384 x 4096 19 / 22
//          64 rows   4096 x 4096 12 / 18, 8192 x 8192 30 / 33, 11008 x 2048 16 / 13,
//                    16384 x 4096 27 / 22, 28672 x 8192 79 / 50, 4096 x 128 5 / 6,
//                    28672 x 128 12 / 7; 4096 x 11008 33 / 41, 8192 x 11008 61 / 41,
//                    2048 x 16384 26 / 55
//          96, 128   96 x 4096 x 11008 50 / 41; 128 x 2048 x 8192 21 / 32, 4096 x 4096
//                    17 / 20, 6144 x 4096 22 / 20, 1024 x 16384 28 / 56
//          256       1024 x 8192 20 / 34, 2048 x 2048 11 / 13, 4096 x 4096 27 / 22,
//                    8192 x 128 12 / 7, 1024 x 11008 41 / 42
//   4-bit, 32 rows   4096 x 4096 6 / 7, 8192 x 8192 13 / 14, 4096 x 11008 15 / 17, 16384 x 4096
//                    10.5 / 10.7, 28672 x 8192 27 / 35, 28672 x 2048 10.5 / 9.6
//          64 rows   4096 x 4096 6.9 / 7.8, 4096 x 8192 11 / 13, 8192 x 8192 16 / 15,
//                    4096 x 2048 6.1 / 5.8, 28672 x 2048 15 / 10; 28672 x 8192 32 / 38, x 4096
//                    20 / 22 (scales in a pass)
//          128       512 x 4096 6 / 7, 2048 x 8192 11 / 12, 4096 x 8192 16 / 13
//          256       1024 x 8192 11 / 12, 2048 x 2048 7 / 6
bool skinny(int64_t M, int64_t N, int64_t K) {
  return K >= 128 && (M <= 32 || (M <= 512 && M * N <= (K <= 8192 ? 1 << 19 : 1 << 18)));
}
bool skinny_mx(int64_t M, int64_t N, int64_t K) {
  return K >= 128 && (M <= 32 || (K <= 8192 && ((M <= 64 && !resident(M, N, K)) ||
                                                (M <= 512 && K >= 4096 && M * N <= 1 << 18))));
}
constexpr int64_t kRowPad = 128;  // rows of 16-bit activations are padded to a tile

int64_t split_row_groups(int64_t M) { return (M + kRowPad - 1) / kRowPad * (kRowPad / 32); }
int64_t split_ksteps(int64_t K) { return (K + 127) / 128 * 2; }

}  // namespace

size_t mxfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M == 1 && K <= mxfp4_gemv_max_k()) return 0;
  if (skinny(M, N, K))
    return K <= mxfp4_skinny_max_k() ? 0 : (size_t)((M + 15) / 16 * ((K + 511) / 512 * 4)) * kMxFragBytes;
  return (size_t)(split_row_groups(M) * split_ksteps(K)) * kMxFragBytes + scale_bytes(N, K);
}

hipError_t launch_mxfp4_gemm(const void* X, int xdtype, const void* codes, const void* scales, int64_t M, int64_t N,
                             int64_t K, void* Y, void* workspace, hipStream_t stream) {
  if (M == 1 && K <= mxfp4_gemv_max_k()) return launch_mxfp4_gemv(X, xdtype, codes, scales, N, K, Y, stream);
  const bool few = skinny(M, N, K);
  if (few && K <= mxfp4_skinny_max_k()) return launch_mxfp4_skinny(X, xdtype, codes, scales, M, N, K, Y, stream);
  const int64_t rg = few ? (M + 15) / 16 : split_row_groups(M), ks = few ? (K + 511) / 512 * 4 : split_ksteps(K);
  uint8_t* const ws = static_cast<uint8_t*>(workspace) + rg * ks * kMxFragBytes;
  const hipError_t e = launch_mxfp4_split(X, M, K, few ? 16 : 32, rg, ks, workspace, few ? nullptr : scales, N, ws, stream);
  if (e != hipSuccess) return e;
  if (few) return launch_mxfp4_skinny(workspace, xdtype, codes, scales, M, N, K, Y, stream);
  return xdtype == 0 ? launch<F16, F16>(workspace, nullptr, codes, ws, M, N, K, Y, stream)
                     : launch<BF16, BF16>(workspace, nullptr, codes, ws, M, N, K, Y, stream);
}

size_t mxfp4_gemm_mx_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return skinny_mx(M, N, K) || resident(M, N, K) ? 0 : scale_bytes(M, K) + scale_bytes(N, K);
}

hipError_t launch_mxfp4_gemm_mx(const void* A, const void* As, const void* W, const void* Ws, int64_t M, int64_t N,
                                int64_t K, int ydtype, void* Y, void* workspace, hipStream_t stream) {
  if (skinny_mx(M, N, K)) return launch_mxfp4_skinny_mx(A, As, W, Ws, M, N, K, ydtype, Y, stream);
  if (!resident(M, N, K)) {
    uint8_t* const ws = static_cast<uint8_t*>(workspace);
    uint8_t* const as = ws + scale_bytes(N, K);
    const hipError_t e = launch_mxfp4_scales(Ws, N, ws, As, M, as, K, stream);
    if (e != hipSuccess) return e;
    As = as;
    Ws = ws;
  }
  return ydtype == 0 ? launch<F16, Mx>(A, As, W, Ws, M, N, K, Y, stream) : launch<BF16, Mx>(A, As, W, Ws, M, N, K, Y, stream);
}

}  // namespace woq
