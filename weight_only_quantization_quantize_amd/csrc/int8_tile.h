// Tiles of products of 8-bit integer matrices: sums over K of a[m, k] w[n, k], exact in
// 32-bit integers, for A [., K] and W [., K] with rows as stored (K a multiple of 16).
//
// Tile.  A group of WM x WN waves computes 32 WM TM x 32 WN TN sums, a wave 32 TM x 32 TN, on
// v_mfma_i32_32x32x32_i8; KG groups of a workgroup share the tile's K and add their sums
// through LDS at the end.
//
// Pipeline.  K goes in stages of 32 KS, two or more of them in LDS, filled by direct loads
// (global_load_lds: no registers, no instructions to write LDS).  A turn multiplies a
// stage.  Before its last units, whose operands are in registers by then, a wave waits until
// its own loads of the next stage are done, meets the others at the barrier, which also says
// that everybody has read this stage, starts the loads of a later stage into its place, and
// reads the next stage's first operands; the units left cover those reads.  The loads are
// written out in assembly because the compiler would wait for all of them before every read
// of LDS; their counter is waited for by hand, and there is no other vector memory access
// inside the loop.  Loads past a row's end repeat its last 16 bytes; the last stage masks
// them on W's side.
//
// What bounds it.  On registers alone the matrix units make 5.0 P op/s of zeros, 3.3 P of
// random codes and, with the LDS reads of a 128 x 64 wave tile beside them, 2.8 P (the
// clock falling with the power, it seems: zeros keep 4.2 P with the same reads).  The products
// reach 2.3 .. 2.4 P (8192 x 8192 x 8192 450 us, a library product 526; 2048 x 11008 x 4096
// 80 .. 85, 104).  LDS is the other limit: a 256 x 256 tile of 8 waves reads 192 KB and takes in
// 64 KB for each 2048 cycles of matrix instructions, 128 bytes a cycle.  Reading operands a
// unit ahead, and past the barrier, took 8192 x 8192 x 8192 from 474 to 450 us; stages
// of 64 K take 498, wave tiles of 128 x 128 on 4 waves 484, and a third stage of W alone
// changes nothing.
//
// LDS layout: a row's 32 KS bytes of a stage are chunks of 16, chunk c at position
// c ^ swizzle(row), so that 16 rows read at one chunk lie in 16 different 16-byte slots of
// the 256-byte bank row.
#pragma once

#include <type_traits>

#include "int8_device.h"

namespace woq {

typedef __attribute__((address_space(3))) uint8_t int8_lds_byte;
__device__ inline uint32_t int8_lds_address(const void* p) { return (uint32_t)(uintptr_t)(const int8_lds_byte*)p; }

// Direct load to LDS: lane l's 16 bytes from base + offset go to to + 16 l.  M0 holds the
// LDS address.  The five wait states cover the write of M0 and a base address that a
// vector instruction wrote just before.  The caller waits for the data.  (The compiler
// reserves M0 and warns of it on a clobber list; it heeds the clobber where it sets M0 for
// itself.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ inline void int8_load_lds(const int8_t* base, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base)
               : "m0", "memory");
}
#pragma clang diagnostic pop
// Until at most N of the wave's vector memory loads are under way and its LDS reads are
// done.
template <int N>
__device__ inline void int8_wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// OCC: waves a SIMD that the registers are shared among.
template <int TM_, int TN_, int WN_, int KS_, int KG_, int NS_, int OCC_ = 2, int WM_ = 2>
struct Int8Tile {
  static constexpr int TM = TM_, TN = TN_, WN = WN_, KS = KS_, KG = KG_, kOccupancy = OCC_, WM = WM_;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves * KG;
  static constexpr int BM = 32 * WM * TM, BN = 32 * WN * TN;
  static constexpr int kRow = 32 * KS;      // bytes of a row's stage
  static constexpr int kChunks = 2 * KS;    // of 16 bytes
  static constexpr int kUnitRows = 1024 / kRow;
  static constexpr int kWUnits = BN / kUnitRows;
  // LDS: NS stages of whole tiles, or all of it where a second workgroup has no place anyway.
  // A tile of few rows has shorter stages, and more of them: it has less to hide its loads
  // behind (a layer of 2048 tokens, where two tiles of three are short: 404 us, 414 without).
  __host__ __device__ static constexpr int stage_bytes(int blocks) { return (32 * WM * blocks + BN) * kRow; }
  static constexpr int kWhole = KG * NS_ * stage_bytes(TM);
  static constexpr int kMost = 159 * 1024;  // of the 160 KB; the rest is the caller's
  static constexpr int kLdsBytes = kWhole > 80 * 1024 && kWhole < kMost ? kMost : kWhole;
  static constexpr int kGroupBytes = kLdsBytes / KG / 1024 * 1024;
  __host__ __device__ static constexpr int stages(int blocks) {
    const int n = blocks == TM ? NS_ : kGroupBytes / stage_bytes(blocks);
    return n > 8 ? 8 : n;
  }
  static constexpr int kWLoads = (kWUnits + kWaves - 1) / kWaves;
  static_assert(kWhole <= 160 * 1024 && KS % 2 == 0);

  template <int TME>
  using Sums = int16v_t[TME][TN];

  __device__ static int swizzle(int row) { return KS == 4 ? (row >> 1) & 7 : (row >> 2) & 3; }

  // The tile's row blocks of 32 go around its WM rows of waves: wave row wm holds the blocks
  // wm, WM + wm, ...  A tile of few rows has blocks at the end that nobody needs, and the
  // work is the same for all waves still.
  __device__ static int row_block(int wave, int i) { return i * WM + wave % WM; }
  // Wave rows of blocks that `rows` rows need, 1 .. TM.
  __device__ static int blocks(int rows) { return rows >= BM ? TM : (rows + 32 * WM - 1) / (32 * WM); }

  // acc[i][j] of the first group's waves: the lane's sums of row 32 row_block(wave, i) +
  // lane % 32 of A and, element e, row 32 (wave / WM TN + j) + 8 (e / 4) + 4 (lane / 32) +
  // e % 4 of W, for the tile's first TME wave rows of blocks; false for the other groups'
  // waves.
  // a_row(r), w_row(r): byte offsets (below 2^32) of the tile's rows from a and w, for
  // every r of the tile.  All threads call; LDS may be used again behind the next barrier.
  template <int TME, class AR, class WR>
  __device__ __forceinline__ static bool multiply(Sums<TME>& acc, uint8_t* __restrict__ lds_all, const int8_t* __restrict__ a,
                                                  AR&& a_row, const int8_t* __restrict__ w, WR&& w_row, int K) {
    constexpr int kAUnits = 32 * WM * TME / kUnitRows, kALoads = (kAUnits + kWaves - 1) / kWaves, kLoads = kALoads + kWLoads;
    constexpr int kStage = stage_bytes(TME), kStages = stages(TME), kAt = 32 * WM * TME * kRow;
    static_assert(kStages >= 2 && kStages * kStage <= kGroupBytes);
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // addresses are worked out for each tile: kept, they spill
    const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = wave_all % kWaves, group = wave_all / kWaves;
    const int wm = wave % WM, wn = wave / WM * TN;
    const int half = lane >> 5, r32 = lane & 31;
    const int chunks = K >> 4;
    const int stages = (chunks + kChunks - 1) / kChunks;
    // K group `group` takes `turns` stages from h0 on; what is missing is missing at the first
    // group's begin (h < 0), so that a short last stage is everybody's last turn
    const int turns = (stages + KG - 1) / KG;
    const int h0 = stages - (KG - group) * turns;
    uint8_t* const lds = lds_all + group * kGroupBytes;
    const uint32_t lds0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)int8_lds_address(lds));

    // Every wave starts the same number of loads a stage: past an operand's units the last
    // one is loaded again, past the last stage that stage.
    auto unit = [&](int j, int units) {
      const int u = wave + kWaves * j;
      return u < units ? u : units - 1;
    };
    uint32_t a_off[kALoads], w_off[kWLoads];
    const int lr = lane / kChunks;
    const int chunk = (lane & (kChunks - 1)) ^ swizzle(lr);
#pragma unroll
    for (int j = 0; j < kALoads; ++j) a_off[j] = a_row(unit(j, kAUnits) * kUnitRows + lr);
#pragma unroll
    for (int j = 0; j < kWLoads; ++j) w_off[j] = w_row(unit(j, kWUnits) * kUnitRows + lr);
    auto issue = [&](int h_, int buf) {
      const int h = h_ < 0 ? 0 : (h_ < stages ? h_ : stages - 1);
      const uint32_t to = lds0 + (uint32_t)(buf * kStage);
      // (the swizzle of a unit's rows: that of its first 1024 / kRow rows, and, of an odd
      // unit of 8 rows, the other half)
      int at[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int c = kChunks * h + (KS == 4 ? chunk ^ (p << 2) : chunk);
        at[p] = 16 * (c < chunks ? c : chunks - 1);
      }
#pragma unroll
      for (int j = 0; j < kALoads; ++j) {
        const int u = unit(j, kAUnits);
        int8_load_lds(a, a_off[j] + (uint32_t)(KS == 4 && (u & 1) ? at[1] : at[0]), to + 1024u * (uint32_t)u);
      }
#pragma unroll
      for (int j = 0; j < kWLoads; ++j) {
        const int u = unit(j, kWUnits);
        int8_load_lds(w, w_off[j] + (uint32_t)(KS == 4 && (u & 1) ? at[1] : at[0]), to + (uint32_t)kAt + 1024u * (uint32_t)u);
      }
    };

    // where the lane's operands of step 0 lie in a stage; step s: bits 5 and 6 flipped by s
    const uint32_t a_at = (uint32_t)((wm * 32 + r32) * kRow + (half ^ swizzle(r32)) * 16);
    const uint32_t w_at = (uint32_t)(kAt + (wn * 32 + r32) * kRow + (half ^ swizzle(r32)) * 16);
#pragma unroll
    for (int i = 0; i < TME; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

    // A unit is row block i of step s: TN matrix instructions.  Operands are read from LDS a
    // unit ahead; the last kTail units of a stage run behind the barrier that ends it, with
    // their operands in registers, and cover the next stage's first reads.
    constexpr int kUnits = KS * TME, kTail = TME < 3 ? 1 : TME - 1, kSlots = kTail + 1;
    static_assert(kUnits % kSlots == 0, "a stage's first unit follows the last one's place");
    int4v_t v[kSlots], wc[2][TN];
    auto read = [&](uint32_t at) { return *reinterpret_cast<const __attribute__((address_space(3))) int4v_t*>(at); };
    auto read_a = [&](uint32_t la, int u) { v[u % kSlots] = read(((la + a_at) ^ (uint32_t)(32 * (u / TME))) + u % TME * WM * 32 * kRow); };
    auto read_w = [&](uint32_t la, int s) {
#pragma unroll
      for (int j = 0; j < TN; ++j) wc[s & 1][j] = read(((la + w_at) ^ (uint32_t)(32 * s)) + j * 32 * kRow);
    };
    // Until stage h's own loads are done, everybody's, and everybody has read the stage
    // before, whose place takes the stage kStages - 1 ahead.
    int buf = 0;  // of stage h
    auto enter = [&](int h) {
      int8_wait_loads<(kStages - 2) * kLoads>();
      __builtin_amdgcn_s_barrier();
      issue(h + kStages - 1, buf == 0 ? kStages - 1 : buf - 1);
    };
    for (int st = 0; st + 1 < kStages; ++st) issue(h0 + st, st);
    enter(h0);
    read_w(lds0, 0);
    read_a(lds0, 0);
    auto turn = [&](int h, auto masked) {
      uint32_t la = lds0 + (uint32_t)(buf * kStage);
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int s = u / TME, i = u % TME;
        if (u == kUnits - kTail) {
          buf = buf + 1 == kStages ? 0 : buf + 1;
          la = lds0 + (uint32_t)(buf * kStage);
          enter(h + 1);
          read_w(la, 0);
          read_a(la, 0);
        }
        if (i == (TME > 1 ? TME - 2 : 0) && s + 1 < KS) read_w(la, s + 1);
        if (u < kUnits - kTail - 1) read_a(la, u + 1);
        if (u == kUnits - kTail - 1)
#pragma unroll
          for (int p = u + 1; p < kUnits; ++p) read_a(la, p);
        if constexpr (decltype(masked)::value) {
          if (i == 0)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) wc[s & 1][j][e] = h * kChunks + 2 * s + half < chunks ? wc[s & 1][j][e] : 0;
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wc[s & 1][j], v[u % kSlots], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (KG > 1 && h < 0)  // what a stage that is not there gave
#pragma unroll
        for (int i = 0; i < TME * TN; ++i) acc[i / TN][i % TN] = int16v_t{};
    };
    const bool rest = stages * kChunks > chunks;
    const int end = h0 + turns - (rest ? 1 : 0);
    for (int h = h0; h < end; ++h) turn(h, std::false_type{});
    if (rest) turn(end, std::true_type{});
    int8_wait_loads<0>();  // none may land in LDS that is another workgroup's by then
    __syncthreads();       // nobody reads operands any more

    if constexpr (KG > 1) {
      // the groups' sums meet in LDS, [wave][tile][lane]
      static_assert(TME * TN * kWaves * 4096 <= kGroupBytes, "a group's sums fit its stages' place");
      int16v_t* const mine = reinterpret_cast<int16v_t*>(lds) + wave * TME * TN * 64 + lane;
      if (group)
#pragma unroll
        for (int i = 0; i < TME * TN; ++i) mine[i * 64] = acc[i / TN][i % TN];
      __syncthreads();
      if (group) return false;
#pragma unroll
      for (int g = 1; g < KG; ++g) {
        const int16v_t* const other = reinterpret_cast<const int16v_t*>(lds_all + g * kGroupBytes) + wave * TME * TN * 64 + lane;
#pragma unroll
        for (int i = 0; i < TME * TN; ++i) acc[i / TN][i % TN] += other[i * 64];
      }
    }
    return true;
  }

  // f(integral_constant blocks(rows)), code of its own for each.
  template <class F>
  __device__ __forceinline__ static void for_blocks(int rows, F&& f) {
    const int n = blocks(rows);
    if constexpr (TM > 4)
      if (n == 4) return f(std::integral_constant<int, 4>{});
    if constexpr (TM > 3)
      if (n == 3) return f(std::integral_constant<int, 3>{});
    if constexpr (TM > 2)
      if (n == 2) return f(std::integral_constant<int, 2>{});
    if constexpr (TM > 1)
      if (n == 1) return f(std::integral_constant<int, 1>{});
    f(std::integral_constant<int, TM>{});
  }
};

// A wave's COLS columns of 32 rows of values, value(row, column block of 4) as a float4_t
// of the lane's row lane % 32, turned through LDS of the wave's own and written in whole
// runs of a row, 16 bytes a lane.  y: of row 0 and the first column; rows, cols: how many
// there are; block b of 4 columns is asked of the half (lane / 32) = b % 2 only.
template <class YT, int COLS, class F>
__device__ inline void int8_store_rows(uint8_t* __restrict__ turn, typename Int8Out<YT>::type* __restrict__ y, int64_t pitch,
                                       int rows, int cols, F&& value) {
  typedef typename Int8Out<YT>::type T;
  constexpr int kSize = (int)sizeof(T), kPitch = COLS * kSize + 16, kLaneCols = 16 / kSize, kRuns = COLS / kLaneCols;
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // as above
  const int half = lane >> 5, r32 = lane & 31;
#pragma unroll
  for (int b = 0; b < COLS / 8; ++b) {
    const float4_t v = value(b);
    T* const to = reinterpret_cast<T*>(turn + r32 * kPitch) + 8 * b + 4 * half;
    if constexpr (kSize == 4) {
      *reinterpret_cast<float4_t*>(to) = v;
    } else {
      *reinterpret_cast<u32x2_t*>(to) = u32x2_t{(uint32_t)Int8Out<YT>::of(v[0]) | (uint32_t)Int8Out<YT>::of(v[1]) << 16,
                                                (uint32_t)Int8Out<YT>::of(v[2]) | (uint32_t)Int8Out<YT>::of(v[3]) << 16};
    }
  }
  asm volatile("" ::: "memory");
#pragma unroll
  for (int q = 0; q < 32 * kRuns / 64; ++q) {
    const int row = (64 * q + lane) / kRuns, c = (64 * q + lane) % kRuns * kLaneCols;
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(turn + row * kPitch + c * kSize);
    if (row < rows && c < cols) {
      T* const to = y + row * pitch + c;
      if (c + kLaneCols <= cols) {
        __builtin_memcpy(to, &v, 16);  // of any alignment: the pitch may be odd
      } else {
        T e[kLaneCols];
        __builtin_memcpy(e, &v, 16);
#pragma unroll
        for (int i = 0; i < kLaneCols; ++i)
          if (c + i < cols) to[i] = e[i];
      }
    }
  }
  asm volatile("" ::: "memory");
}

}  // namespace woq
