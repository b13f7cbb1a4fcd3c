// A layer of gated experts with 8-bit integer weights, for tokens that are routed already:
//   q, a   = the codes and scales of X's rows (int8_quantize)
//   g, u   = (acc a[t]) s_up[e, .] of the gate and the up rows of up[e], acc = sum_k q[t, k] up[e, ., k]
//   h      = silu(g) u, silu(g) = g / (1 + exp(-g)), fp32; quantised by rows again: p, b
//   y[t,c] = (acc b) s_down[e, .],  acc = sum_i p[i] down[e, ., i]
//   Y[t]   = sum over the token's choices c of weights[t, c] y[t, c], rounded once
// A choice whose expert is none of 0 .. E - 1 is left out.
//
// Launches: `prepare` quantizes the rows of X and, in its first workgroup, sorts the choices
// by expert into rows and cuts each expert's rows into tiles; `up` and `down` are tile
// products (int8_tile.h) over those tiles; h's rows are quantized between them; `combine`
// adds up.  The rows' order in the plan changes no result: every row is computed by itself.
//
// One token has two launches of its own (int8_moe_row.hip).
//
// Work of the products.  Experts' row counts differ, and a tile of few rows is cheap
// (int8_tile.h: it multiplies its own blocks of rows only), so tiles are taken, not dealt: a
// workgroup a compute unit's place takes tile after tile, those of the experts with the most
// rows first.  With many tokens the weights' bytes bound the products as much as the matrix
// units do (a dense product of 256 rows with as many weight bytes takes 165 us, one with few
// weights 115 .. 130), so an expert's weights should come out of HBM once: its row tiles of
// one column tile are neighbours in the run of one XCD, are multiplied at the same time and
// share the weights in its L2.  The column tiles go around the XCDs, which so have the same
// work.  2048 tokens of 32 experts 4096 x 2048, four each, whole layer: 389 us when this was
// chosen; each XCD an eighth of all tiles, experts in a row, 412, with the idle ones helping
// out 417.
//
// An expert's second tile reads the weights again, so tiles of many rows are 320 high, all
// that registers and LDS hold, and an expert's rows are spread evenly over its tiles, in whole
// row blocks.  The same layer, routed evenly (unevenly: logits with a normal bias for each
// expert), T tokens, tiles of 256 rows with a short last one before it:
//   T     1500         2048         3000         4096
//   now   305 (348)    356 (385)    478 (498)    602 (643) us
//   256   305 (331)    382 (430)    500 (513)    642 (659)
// (320 rows with a short last tile: 550 for 3000 tokens; 256 rows, even: 384 for 2048.)
#include "int8_rows.h"
#include "int8_tile.h"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kMaxExperts = 512;
constexpr int kXcds = 8;
constexpr int kRowBlock = 64;  // tiles' rows are multiplied by as many (int8_tile.h; 32 of each of two waves)

// Up to BM rows of an expert, whose rank by rows is `rank`.
struct Tile {
  int expert, row, count, rank;
};
// Row tiles; how many items of each XCD's run were taken so far (beside the first ones, which
// are dealt), of up and of down.
struct Plan {
  int tiles;
  int taken[2][kXcds];
};

// One workgroup of at least 64 threads.  where [T top_k]: a choice's row, -1 of none; token [rows].
__device__ void int8_moe_plan(const int32_t* __restrict__ experts, int choices, int top_k, int E, int BM, Plan* __restrict__ plan,
                              Tile* __restrict__ tiles, int* __restrict__ where, int* __restrict__ token) {
  __shared__ int count[kMaxExperts], first[kMaxExperts], by_rank[kMaxExperts];
  const int threads = blockDim.x;
  for (int e = threadIdx.x; e < E; e += threads) count[e] = 0;
  if (threadIdx.x < 2 * kXcds) plan->taken[threadIdx.x / kXcds][threadIdx.x % kXcds] = 0;
  __syncthreads();
  // the choices, 8 a thread on their way at a time
  auto each = [&](auto f) {
    for (int i0 = threadIdx.x; i0 < choices; i0 += 8 * threads) {
      int e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = experts[i0 + j * threads < choices ? i0 + j * threads : i0];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + j * threads < choices) f(i0 + j * threads, e[j]);
    }
  };
  each([&](int, int e) {
    if (e >= 0 && e < E) atomicAdd(&count[e], 1);
  });
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += threads) {
    const int n = count[e];
    int rank = 0;
    for (int o = 0; o < E; ++o) rank += count[o] > n || (count[o] == n && o < e);
    by_rank[rank] = e;
  }
  __syncthreads();
  if (threadIdx.x < 64) {  // rows and row tiles before each rank
    const int lane = threadIdx.x;
    int rows = 0, of = 0;
    for (int r0 = 0; r0 < E; r0 += 64) {
      const int r = r0 + lane, e = by_rank[r < E ? r : 0], n = r < E ? count[e] : 0;
      // an expert's tiles are of one height, in whole row blocks, but for the last one
      const int least = (n + BM - 1) / BM, height = n ? (n + kRowBlock * least - 1) / (kRowBlock * least) * kRowBlock : BM;
      const int m = (n + height - 1) / height;
      int a = n, b = m;
      for (int off = 1; off < 64; off <<= 1) {
        const int p = __shfl_up(a, off, 64), q = __shfl_up(b, off, 64);
        if (lane >= off) a += p, b += q;
      }
      if (r < E) {
        const int row = rows + a - n;
        first[e] = row;
        for (int i = 0; i < m; ++i)
          tiles[of + b - m + i] = Tile{e, row + i * height, n - i * height < height ? n - i * height : height, r};
      }
      rows += __shfl(a, 63, 64);
      of += __shfl(b, 63, 64);
    }
    if (lane == 0) plan->tiles = of;
  }
  __syncthreads();
  each([&](int i, int e) {
    int row = -1;
    if (e >= 0 && e < E) {
      row = atomicAdd(&first[e], 1);
      token[row] = i / top_k;
    }
    where[i] = row;
  });
}

template <class XT, int STEPS>
__global__ __launch_bounds__(kRowMaxWaves * 64) void int8_moe_prepare_kernel(
    const void* __restrict__ X, int64_t T, int H, int W, int rounds, int8_t* __restrict__ codes, float* __restrict__ scales,
    const int32_t* __restrict__ experts, int top_k, int E, int BM, Plan* __restrict__ plan, Tile* __restrict__ tiles,
    int* __restrict__ where, int* __restrict__ token) {
  if (blockIdx.x == 0)
    int8_moe_plan(experts, (int)T * top_k, top_k, E, BM, plan, tiles, where, token);
  else
    int8_quantize_rows<XT, kNone, STEPS>(X, nullptr, T, H, W, rounds, (int64_t)blockIdx.x - 1, codes, scales);
}

// The outputs of a tile's sums: h of its gate and up columns, or its products.
template <bool UP, class C, int TME>
__device__ __forceinline__ void finish(const typename C::template Sums<TME>& acc, uint8_t* __restrict__ lds, const float* __restrict__ sa,
                                       const float* __restrict__ s, const int* __restrict__ token, const Tile& tile, int N, int n0,
                                       float* __restrict__ out) {
  auto clamped = [&](int r) { return r < tile.count ? r : tile.count - 1; };
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // addresses are worked out for each tile: kept, they spill
  const int half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kCols = UP ? 16 * C::TN : 32 * C::TN;
  constexpr int kTurn = 32 * (kCols * 4 + 16) + kCols * 8;
  static_assert(C::kWaves * kTurn <= C::kGroupBytes, "the turn fits the stages' place");
  static_assert(32 * C::WM == kRowBlock && C::BM % kRowBlock == 0, "tiles' heights are whole row blocks");
  static_assert(!UP || C::TN % 2 == 0, "a wave has gate and up columns");
  const int n1 = n0 + wave / C::WM * kCols;
  uint8_t* const turn = lds + wave * kTurn;
  float* const cols = reinterpret_cast<float*>(turn + 32 * (kCols * 4 + 16));
  for (int c = lane; c < kCols; c += 64) {
    const int n = n1 + c < N ? n1 + c : N - 1;
    cols[c] = s[n];
    if (UP) cols[kCols + c] = s[N + n];
  }
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < TME; ++i) {
    const int m = 32 * C::row_block(wave, i), r = clamped(m + (lane & 31));
    if (m >= tile.count) break;
    const float f = sa[UP ? token[tile.row + r] : tile.row + r];
    int8_store_rows<F32, kCols>(turn, out + (int64_t)(tile.row + m) * N + n1, N, tile.count - m, N - n1, [&](int b) {
      const float4_t c = *reinterpret_cast<const float4_t*>(cols + 8 * b + 4 * half);
      float4_t v;
      if constexpr (UP) {
        const float4_t d = *reinterpret_cast<const float4_t*>(cols + kCols + 8 * b + 4 * half);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float g = (float)acc[i][b / 4 * 2][4 * (b % 4) + e] * f * c[e];
          const float u = (float)acc[i][b / 4 * 2 + 1][4 * (b % 4) + e] * f * d[e];
          v[e] = int8_gated(g, u);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][b / 4][4 * (b % 4) + e] * f * c[e];
      }
      return v;
    });
  }
}

// UP: A = X's codes, gathered; W's tile is blocks of 32 gate rows and the 32 up rows of the
// same columns in turn.  Else A = h's codes.  ntiles: of columns of h (of y).
template <bool UP, class C>
__global__ __launch_bounds__(C::kThreads, C::kOccupancy) void int8_moe_product_kernel(
    const int8_t* __restrict__ A, const float* __restrict__ sa, const int8_t* __restrict__ W, const float* __restrict__ sw,
    Plan* __restrict__ plan, const Tile* __restrict__ tiles, const int* __restrict__ token, int K, int N, int ntiles,
    float* __restrict__ out) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kLdsBytes];
  __shared__ int next;
  // item k of XCD x is number x + 8 k of the pairs of a row tile and a column tile; large
  // tiles' columns are counted as a multiple of 8, which keeps a column tile on its XCD
  const int x = (int)blockIdx.x % kXcds, own = (int)gridDim.x / kXcds;  // workgroups of an XCD: their first items are dealt
  const int columns = C::TM > 1 ? (ntiles + kXcds - 1) / kXcds * kXcds : ntiles, items = plan->tiles * columns;
  for (int item = (int)blockIdx.x; item < items;) {
    const Tile tile = tiles[item / columns];
    const int nt = (item % columns + (C::TM > 1 ? tile.rank : 0)) % columns;
    const int n0 = nt * (UP ? C::BN / 2 : C::BN);
    const int rows = UP ? 2 * N : N;  // of an expert's weights
    const int8_t* const w = W + (int64_t)tile.expert * rows * K;
    const float* const s = sw + (int64_t)tile.expert * rows;
    auto clamped = [&](int r) { return r < tile.count ? r : tile.count - 1; };
    int after = 0;
    if (threadIdx.x == 0) after = atomicAdd(&plan->taken[UP ? 0 : 1][x], 1);  // on its way meanwhile
    if (nt < ntiles)
      C::for_blocks(tile.count, [&](auto blocks) {
        constexpr int kBlocks = decltype(blocks)::value;
        typename C::template Sums<kBlocks> acc;
        const bool mine = C::template multiply<kBlocks>(
            acc, lds, UP ? A : A + (int64_t)tile.row * K,
            [&](int r) { return (uint32_t)(UP ? token[tile.row + clamped(r)] : clamped(r)) * (uint32_t)K; }, w,
            [&](int r) {
              const int n = UP ? n0 + (r >> 6) * 32 + (r & 31) : n0 + r;
              return ((uint32_t)(n < N ? n : N - 1) + (UP && (r & 32) ? (uint32_t)N : 0u)) * (uint32_t)K;
            },
            K);
        if (mine) finish<UP, C, kBlocks>(acc, lds, sa, s, token, tile, N, n0, out);
      });
    __syncthreads();  // `next` and the LDS were read
    if (threadIdx.x == 0) next = after;
    __syncthreads();
    item = x + kXcds * (own + next);
  }
}

// Y[t] = the sum of its choices' rows of `products`, weighted, in the order of choice.
template <class YT>
__global__ __launch_bounds__(256) void int8_moe_combine_kernel(const float* __restrict__ products, const int* __restrict__ where,
                                                               const float* __restrict__ weights, int T, int H, int top_k,
                                                               uint16_t* __restrict__ Y) {
  const int n = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 4;
  if (n >= H) return;
  for (int t = (int)blockIdx.y; t < T; t += (int)gridDim.y) {
    float4_t v = {};
    for (int c = 0; c < top_k; ++c) {
      const int row = where[(int64_t)t * top_k + c];
      if (row < 0) continue;
      const float w = weights[(int64_t)t * top_k + c];
      const float4_t p = *reinterpret_cast<const float4_t*>(products + (int64_t)row * H + n);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = fmaf(w, p[e], v[e]);
    }
    const uint32_t lo = (uint32_t)YT::from_f32(v[0]) | (uint32_t)YT::from_f32(v[1]) << 16;
    const uint32_t hi = (uint32_t)YT::from_f32(v[2]) | (uint32_t)YT::from_f32(v[3]) << 16;
    *reinterpret_cast<u32x2_t*>(Y + (int64_t)t * H + n) = u32x2_t{lo, hi};
  }
}

typedef Int8Tile<1, 2, 2, 4, 1, 3> Small;
typedef Int8Tile<5, 2, 4, 4, 1, 2> Large;

// Tiles of rows, at most: one for each expert that is taken and one for each further BM.
int64_t most_tiles(int64_t choices, int64_t E, int64_t BM) { return (choices < E ? choices : E) + choices / BM; }
// Small tiles stream the weights with the least work for rows that are not there, and there
// are enough of them where the layer is small; large ones read LDS and the weights least.
// Large ones are taken where the up product has one for every compute unit and an expert has
// more than 56 rows in the mean, or 128 and for three compute units of four.  Of 49 layers (H
// 512 .. 4096, I 256 .. 4096, 4 .. 128 experts, 8 .. 4096 rows an expert), routed evenly and
// unevenly, the choice takes 1.2% more than the faster tile in the mean, 15% at most.  Small,
// large: H 4096, I 2048, 32 experts, 48, 64 and 128 rows: 201, 213 us; 221, 225; 306, 273; H
// 1024, I 512, 8 experts, 128, 1024 and 4096 rows: 29, 63; 86, 117; 248, 231.
int64_t tile_rows(int64_t T, int64_t I, int64_t E, int64_t top_k) {
  const int64_t choices = T * top_k, rows = choices / E;
  const int64_t tiles = (choices < E ? choices : E) * ((rows + Large::BM - 1) / Large::BM) * ((2 * I + Large::BN - 1) / Large::BN);
  return (rows > 56 && tiles >= 256) || (rows >= 128 && tiles >= 192) ? Large::BM : Small::BM;
}

struct Layout {
  size_t codes, scales, plan, tiles, where, token, h, h_codes, h_scales, products, bytes;
};
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
Layout layout(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k) {
  const size_t rows = (size_t)(T * top_k);
  Layout l;
  l.codes = 0;
  l.scales = up256((size_t)(T * H));
  l.plan = up256(l.scales + (size_t)T * 4);
  l.tiles = l.plan + 256;
  l.where = up256(l.tiles + (size_t)most_tiles(T * top_k, E, tile_rows(T, I, E, top_k)) * sizeof(Tile));
  l.token = up256(l.where + rows * 4);
  l.h = up256(l.token + rows * 4);
  l.h_codes = up256(l.h + rows * (size_t)I * 4);
  l.h_scales = up256(l.h_codes + rows * (size_t)I);
  l.products = up256(l.h_scales + rows * 4);
  l.bytes = l.products + rows * (size_t)H * 4;
  return l;
}

}  // namespace

int int8_moe_max_experts() { return kMaxExperts; }

size_t int8_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k) {
  if (T == 1 && int8_moe_row_supported(H, I, top_k)) return (size_t)(top_k * I) * 4;
  return layout(T, H, I, E, top_k).bytes;
}

hipError_t launch_int8_moe(const void* X, int xdtype, const int32_t* experts, const float* weights, const void* up,
                           const float* up_scales, const void* down, const float* down_scales, int64_t T, int64_t H, int64_t I,
                           int64_t E, int top_k, void* Y, void* workspace, hipStream_t stream) {
  if (T == 1 && int8_moe_row_supported(H, I, top_k))
    return launch_int8_moe_row(X, xdtype, experts, weights, up, up_scales, down, down_scales, H, I, E, top_k, Y, workspace, stream);
  const Layout l = layout(T, H, I, E, top_k);
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  const int64_t choices = T * top_k, BM = tile_rows(T, I, E, top_k);
  Plan* const plan = reinterpret_cast<Plan*>(ws + l.plan);
  Tile* const tiles = reinterpret_cast<Tile*>(ws + l.tiles);
  int* const where = reinterpret_cast<int*>(ws + l.where);
  int* const token = reinterpret_cast<int*>(ws + l.token);
  float* const h = reinterpret_cast<float*>(ws + l.h);
  float* const products = reinterpret_cast<float*>(ws + l.products);
  float* const h_scales = reinterpret_cast<float*>(ws + l.h_scales);
  float* const x_scales = reinterpret_cast<float*>(ws + l.scales);
  const Int8RowsPlan p = int8_rows_plan(T, H);
  auto prepare = [&](auto tag) {
    using XT = decltype(tag);
    auto* const f = p.per <= 1 ? int8_moe_prepare_kernel<XT, 1> : (p.per <= 2 ? int8_moe_prepare_kernel<XT, 2> : int8_moe_prepare_kernel<XT, 4>);
    f<<<p.groups + 1, (unsigned)p.threads(), 0, stream>>>(X, T, (int)H, p.W, p.rounds(), reinterpret_cast<int8_t*>(ws + l.codes), x_scales,
                                                          experts, top_k, (int)E, (int)BM, plan, tiles, where, token);
    return hipGetLastError();
  };
  hipError_t e = xdtype == 0 ? prepare(F16{}) : prepare(BF16{});
  if (e != hipSuccess) return e;
  const int64_t mt = most_tiles(choices, E, BM);
  auto product = [&](auto is_up, auto tag, const void* a, const float* sa, const void* w, const float* sw, int64_t K, int64_t N,
                     float* out) {
    using C = decltype(tag);
    constexpr bool kUp = decltype(is_up)::value;
    constexpr int kCols = kUp ? C::BN / 2 : C::BN;
    const int64_t nt = (N + kCols - 1) / kCols, most = (mt * nt + kXcds - 1) / kXcds * kXcds;
    // the workgroups that the compute units have room for
    constexpr int64_t kRoom = 256 * (C::kLdsBytes <= 80 * 1024 ? 2 : 1);
    int8_moe_product_kernel<kUp, C><<<(unsigned)(most < kRoom ? most : kRoom), C::kThreads, 0, stream>>>(
        static_cast<const int8_t*>(a), sa, static_cast<const int8_t*>(w), sw, plan, tiles, token, (int)K, (int)N, (int)nt, out);
    return hipGetLastError();
  };
  auto products_of = [&](auto tag) {
    hipError_t e = product(std::true_type{}, tag, ws + l.codes, x_scales, up, up_scales, H, I, h);
    if (e != hipSuccess) return e;
    e = launch_int8_quantize(h, 2, nullptr, false, choices, I, ws + l.h_codes, h_scales, stream);
    if (e != hipSuccess) return e;
    return product(std::false_type{}, tag, ws + l.h_codes, h_scales, down, down_scales, I, H, products);
  };
  e = BM == Small::BM ? products_of(Small{}) : products_of(Large{});
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((H + 1023) / 1024), (unsigned)(T < 65535 ? T : 65535));
  auto* const f = xdtype == 0 ? int8_moe_combine_kernel<F16> : int8_moe_combine_kernel<BF16>;
  f<<<grid, 256, 0, stream>>>(products, where, weights, (int)T, (int)H, top_k, static_cast<uint16_t*>(Y));
  return hipGetLastError();
}

}  // namespace woq
