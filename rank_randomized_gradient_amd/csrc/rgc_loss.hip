// A linear layer and its softmax cross entropy over a large vocabulary,
// without keeping the logits, and the gradient that feeds the layer's input
// and its sketch. W: V x k, a row per vocabulary entry; X: T x k.
//
//   z = X W^T,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,y(t)
//   D_tv = g_t (exp(z_tv - lse_t) - [v = y(t)])
//   dX = D W,  C += D^T XP
//
// Tokens whose target lies outside 0 .. V-1 are ignored: no loss and a zero
// row of D.
//
// Forward: every 256 x 256 tile of z is reduced in registers to its rows'
// maxima and sums of exponentials; a second launch joins the tiles of a row.
// Backward: the vocabulary goes by in pieces. A piece's D is formed from z
// again (z costs 2 T V k operations a second time; keeping it would cost 2 T V
// bytes and more), written to the workspace, and used twice from there while it
// is in the last-level cache: D W, added to dX in fp32, and D^T XP, added to the
// sketch by the sketch's own accumulation.
//
// D is kept as two bf16 terms, D = hi + lo (each rounding leaves at most 2^-8 of
// what it rounds, so the pair is off by 2^-17 of D at most), and both products
// take both. One term would do where the softmax is flat, but not for a token
// whose mass lies on a few entries with rows of W near each other: their large
// entries of D cancel in dX, and 2^-8 of each does not (D of +-1/2 on two rows 5%
// apart: dX off by up to 8% in one term, by its own rounding in two). A tile of
// dX takes 128 tokens, their hi and lo as its 256 rows, and adds the two halves
// of its sums in its registers. For the sketch the terms are stacked along the
// tokens: C += [hi; lo]^T [XP; XP] is one accumulation over 2 T tokens.
// What the terms leave of the targets' entries, by far the largest of a flat
// softmax's D (of the order of g, the others of g / V), is kept in fp32, one value
// a token, and added where it costs little: rest_t W_y(t) to dX when it is
// rounded, and rest_t XP_t to C's row y(t) in a last launch. Up to 128 tokens
// one tile holds them all, and adds its rows of the sketch itself, from D in fp32.
//
// Bound by MFMA: 2 T V k operations for the loss, 6 T V k + 4 T V r more for the
// gradient. Where dX has few tiles (few tokens), each is split over K among
// several workgroups, which add into slabs of their own; a last launch adds
// the slabs and rounds. All sums have a fixed order.
#include "rgc_gemm_tile.hpp"

namespace rgc {
namespace {

constexpr int64_t kCeMaxVocab = int64_t(1) << 24;
constexpr int kCeDown = 8;        // tile rows walked together
constexpr int kCeMaxSplit = 128;
constexpr double kCeSmallRate = 0.6;  // a small tile's rate beside a large one's
constexpr float kLog2e = 1.4426950408889634f;

// The logits' tiles of a launch: `large` 256 x 256 ones, which cover the first
// `split` rows of the piece, then small ones for the rest.
struct CeGrid {
  int64_t large, split;
  int64_t ntiles;  // columns of tiles, large and small
};

struct CeArgs {
  const uint16_t* X;
  const uint16_t* W;   // the piece's first row
  const int64_t* targets;
  int64_t ldx, ldw;
  int64_t T, V, k;     // V: rows of the piece
  int64_t v0;          // vocabulary index of the piece's first row
  int64_t vocab;       // rows of the whole vocabulary
  CeGrid grid;
  float2* part;        // forward: (maximum, sum) of each tile row, [tile column][token]
  float* zt;           // forward: the target's logit
  const float* lse;    // backward
  const float* grad;
  uint16_t* hi;        // backward: T x ldd, bf16
  uint16_t* lo;        // or null: nothing takes D from here
  float* rest;         // with lo: D - hi - lo at each token's target
  int64_t ldd;
  float* C;            // few tokens: the sketch's rows of the piece, added to here; else null
  const uint16_t* XP;
  int r;
};

typedef GtTile<8, 4, 2, false> LargeTile;   // 256 x 256
typedef GtTile<4, 2, 4, false> SmallTile;   // 128 x 128
// 64 x 128, for few tokens: three stages, so that two workgroups share a compute
// unit, one's epilogue under the other's product. 64 x 50000 x 1024: D of rank 128
// 49 us with one workgroup on five stages, 40 us so; the forward 23 and 19 us.
typedef GtTile<2, 2, 3, false> FlatTile;
// 128 x 128 on two stages, two workgroups to a compute unit: for a launch of small
// tiles alone that gives every compute unit more than one (pair_tiles).
typedef GtTile<4, 2, 2, false> PairTile;
static_assert(SmallTile::kLds <= LargeTile::kLds, "one LDS array serves the tiles of a launch");

// What an epilogue needs of a tile's rows, fetched before the product.
struct CeRows {
  float lse[kGtTile], grad[kGtTile];
  int at[kGtTile];  // the target's column in the tile; -1: elsewhere; -2: an ignored token
};

template <typename Tile>
__device__ __forceinline__ void load_rows(const CeArgs& a, int64_t m0, int64_t n0, bool backward, CeRows* r) {
  const int row = threadIdx.x;
  if (row >= Tile::kRows) return;
  const bool live = m0 + row < a.T;
  const int64_t y = live ? a.targets[m0 + row] : -1, c = y - a.v0 - n0;
  r->at[row] = y < 0 || y >= a.vocab ? -2 : c >= 0 && c < Tile::kCols ? (int)c : -1;
  if (backward) {
    r->lse[row] = live ? a.lse[m0 + row] : 0.f;
    r->grad[row] = live ? a.grad[m0 + row] : 0.f;
  }
}

// exp(x); below 2^-126 it is zero.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// The tile of rows m0 .. and columns n0 .. of z, reduced to slot `column` of its rows.
template <int MI, int NI, int STAGES>
__device__ __forceinline__ void forward_tile(const CeArgs& a, int64_t m0, int64_t n0, int64_t column, char* smem, CeRows* rows) {
  typedef GtTile<MI, NI, STAGES, false> Tile;
  load_rows<Tile>(a, m0, n0, false, rows);
  Tile t;
  t.init(a.X + m0 * a.ldx, a.ldx, a.W + n0 * a.ldw, a.ldw, a.T - m0, a.V - n0, a.k, smem);
  t.run();

  const int g = t.lane >> 4, li = t.lane & 15, wm = t.wave & 1, wn = t.wave >> 1;
  float* sums = reinterpret_cast<float*>(smem);  // [row][wn]: maximum, sum
  const int first = 16 * NI * wn + 4 * g;
  const int width = (int)(a.V - n0 < Tile::kCols ? a.V - n0 : Tile::kCols);
#pragma unroll
  for (int mt = 0; mt < MI; ++mt) {
    const int row = 16 * MI * wm + 16 * mt + li;
    const int at = rows->at[row] - first;
    if (__builtin_expect(width < Tile::kCols, 0)) {
#pragma unroll
      for (int nt = 0; nt < NI; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (first + 16 * nt + e >= width) t.acc[mt][nt][e] = -INFINITY;
    }
    if (__any(at >= 0 && at < 16 * NI)) {
#pragma unroll
      for (int nt = 0; nt < NI; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * nt + e == at) a.zt[m0 + row] = t.acc[mt][nt][e];
    }
    float top = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NI; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, t.acc[mt][nt][e]);
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const float base = top == -INFINITY ? 0.f : top;
    float s = 0.f;
#pragma unroll
    for (int nt = 0; nt < NI; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s += fast_exp(t.acc[mt][nt][e] - base);
    s += __shfl_xor(s, 16, 64);
    s += __shfl_xor(s, 32, 64);
    if (g == 0) {
      sums[8 * row + 2 * wn] = top;
      sums[8 * row + 2 * wn + 1] = s;
    }
  }
  __syncthreads();
  const int row = threadIdx.x;
  if (row < Tile::kRows && m0 + row < a.T) {
    float top = sums[8 * row], s = 0.f;
#pragma unroll
    for (int w = 1; w < 4; ++w) top = fmaxf(top, sums[8 * row + 2 * w]);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < 4; ++w) s += sums[8 * row + 2 * w + 1] * fast_exp(sums[8 * row + 2 * w] - base);
    a.part[column * a.T + m0 + row] = make_float2(top, s);
  }
}

// Joins a token's tiles: a wave per token, lane l taking every 64th tile from
// l, then the lanes' maxima and sums by a xor butterfly. The sixteen tokens of
// a workgroup share the lines of their partial sums.
__global__ __launch_bounds__(1024) void ce_finish_kernel(CeArgs a, float* loss, float* lse) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 6);
  if (t >= a.T) return;
  float top = -INFINITY, s = 0.f;
#pragma unroll 4
  for (int64_t j = lane; j < a.grid.ntiles; j += 64) {
    const float2 p = a.part[j * a.T + t];
    const float m = fmaxf(top, p.x), base = m == -INFINITY ? 0.f : m;
    s = s * fast_exp(top - base) + p.y * fast_exp(p.x - base);
    top = m;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const float x = __shfl_xor(top, off, 64), y = __shfl_xor(s, off, 64);
    const float m = fmaxf(top, x), base = m == -INFINITY ? 0.f : m;
    s = s * fast_exp(top - base) + y * fast_exp(x - base);
    top = m;
  }
  if (lane == 0) {
    const float l = top + logf(s);
    const int64_t y = a.targets[t];
    lse[t] = l;
    loss[t] = y >= 0 && y < a.vocab ? l - a.zt[t] : 0.f;
  }
}

// R rows and four ranks of C for a thread, the tokens in order.
template <int R>
__device__ __forceinline__ void sketch_rows(float* C, int r, const float* d, int cols, const uint2* xp, int T, int width) {
  const int quads = r / 4, quad = threadIdx.x % quads, part = threadIdx.x / quads, parts = kGtThreads / quads;
  if (part >= parts) return;
  for (int row0 = R * part; row0 < width; row0 += R * parts) {
    f32x4_t sum[R];
#pragma unroll
    for (int i = 0; i < R; ++i) sum[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < T; ++k) {
      const uint2 x = xp[k * quads + quad];
      const f32x4_t w = {__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u), __uint_as_float(x.y << 16),
                         __uint_as_float(x.y & 0xFFFF0000u)};
      float v[R];
#pragma unroll
      for (int i = 0; i < R; ++i) v[i] = d[k * cols + row0 + i];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[i][e] = __builtin_fmaf(v[i], w[e], sum[i][e]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (row0 + i < width) *reinterpret_cast<f32x4_t*>(C + (int64_t)(row0 + i) * r + 4 * quad) += sum[i];
  }
}

// C's rows of a tile += D^T XP, for the tile that holds all T tokens: no partial
// sums to join and no second term of D, which is taken in fp32 from the registers
// by way of LDS. As many neighbouring rows to a thread as give the 512 threads
// the tile's 128 rows in one pass (above rank 64 eight, for fewer LDS reads).
template <int MI, int NI, typename Tile>
__device__ __forceinline__ void sketch_tile(const CeArgs& a, const Tile& t, int64_t n0, int width, char* smem,
                                            const CeRows* rows) {
  constexpr int kCols = Tile::kCols;
  const int g = t.lane >> 4, li = t.lane & 15, wm = t.wave & 1, wn = t.wave >> 1;
  const int T = (int)a.T, quads = a.r / 4;
  float* d = reinterpret_cast<float*>(smem);  // [token][column]
  uint2* xp = reinterpret_cast<uint2*>(smem + 4 * Tile::kRows * kCols);  // [token][quad]
  static_assert(4 * Tile::kRows * kCols + 2 * Tile::kRows * 256 <= Tile::kLds, "D and XP of a tile in LDS");
#pragma unroll
  for (int mt = 0; mt < MI; ++mt)
#pragma unroll
    for (int nt = 0; nt < NI; ++nt)
      *reinterpret_cast<f32x4_t*>(d + (16 * MI * wm + 16 * mt + li) * kCols + 16 * NI * wn + 16 * nt + 4 * g) = t.acc[mt][nt];
#pragma unroll 4
  for (int i = threadIdx.x; i < T * quads; i += kGtThreads) {
    const uint2 x = reinterpret_cast<const uint2*>(a.XP)[i];
    const bool live = rows->at[i / quads] != -2;  // zeros for the ignored, whatever their rows hold
    xp[i] = make_uint2(live ? x.x : 0u, live ? x.y : 0u);
  }
  __syncthreads();
  float* C = a.C + n0 * a.r;
  if (a.r > 64) sketch_rows<8>(C, a.r, d, kCols, xp, T, width);
  else if (a.r > 16) sketch_rows<4>(C, a.r, d, kCols, xp, T, width);
  else sketch_rows<1>(C, a.r, d, kCols, xp, T, width);
  __syncthreads();
}

// A piece's D, hi and lo: T x ldd each, zero in the columns behind the piece.
// The tile's bf16 values are laid out in LDS first, so that they are stored in
// whole rows (16-byte chunk q of row t at place q ^ (t % 16)). The
// lo pass forms D - hi from the fp32 values, which stay in the registers. Without
// lo (a fused sketch and no dX) nothing is stored.
template <int MI, int NI, int STAGES>
__device__ __forceinline__ void d_tile(const CeArgs& a, int64_t m0, int64_t n0, char* smem, CeRows* rows) {
  typedef GtTile<MI, NI, STAGES, false> Tile;
  constexpr int kRowChunks = Tile::kCols / 8;  // 16-byte chunks of a row
  load_rows<Tile>(a, m0, n0, true, rows);
  Tile t;
  t.init(a.X + m0 * a.ldx, a.ldx, a.W + n0 * a.ldw, a.ldw, a.T - m0, a.V - n0, a.k, smem);
  t.run();

  const int g = t.lane >> 4, li = t.lane & 15, wm = t.wave & 1, wn = t.wave >> 1;
  const int first = 16 * NI * wn + 4 * g;
  const int width = (int)(a.V - n0 < Tile::kCols ? a.V - n0 : Tile::kCols);
#pragma unroll
  for (int mt = 0; mt < MI; ++mt) {
    const int row = 16 * MI * wm + 16 * mt + li;
    const int target = rows->at[row], at = target - first;
    const float lse = rows->lse[row], gr = rows->grad[row];
#pragma unroll
    for (int nt = 0; nt < NI; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = fast_exp(t.acc[mt][nt][e] - lse) * gr;
        t.acc[mt][nt][e] = target == -2 ? 0.f : p;
      }
    if (__any(at >= 0 && at < 16 * NI)) {
#pragma unroll
      for (int nt = 0; nt < NI; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * nt + e == at) t.acc[mt][nt][e] -= gr;
    }
    if (__builtin_expect(width < Tile::kCols, 0)) {
#pragma unroll
      for (int nt = 0; nt < NI; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (first + 16 * nt + e >= width) t.acc[mt][nt][e] = 0.f;
    }
  }
  if constexpr (MI <= 4 && STAGES > 2) {  // (two stages leave no LDS for it)
    if (a.C) sketch_tile<MI, NI>(a, t, n0, width, smem, rows);
  }
  if (!a.lo) return;
  RGC_LDS char* lds = (RGC_LDS char*)smem;
  uint32_t to[NI];  // this lane's places in the row of mt = 0
#pragma unroll
  for (int nt = 0; nt < NI; ++nt)
    to[nt] = (uint32_t)(16 * (kRowChunks * (16 * MI * wm + li) + ((2 * NI * wn + 2 * nt + (g >> 1)) ^ li)) + 8 * (g & 1));
  const int row0 = threadIdx.x / kRowChunks, q = (threadIdx.x % kRowChunks) ^ (row0 & 15);
  constexpr int kRowsAtOnce = kGtThreads / kRowChunks;  // a multiple of 16: q holds for every pass
  static_assert(kRowsAtOnce % 16 == 0, "rows of a pass");
#pragma unroll 1
  for (int term = 0; term < 2; ++term) {
    if (term) __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MI; ++mt)
#pragma unroll
      for (int nt = 0; nt < NI; ++nt) {
        const f32x4_t d = t.acc[mt][nt];
        const u32x2v_t h = {f32x2_to_bf16x2_rne(d[0], d[1]), f32x2_to_bf16x2_rne(d[2], d[3])};
        // what the term leaves, exact: it is the value's leading bits
        t.acc[mt][nt] = d - f32x4_t{__uint_as_float(h.x << 16), __uint_as_float(h.x & 0xFFFF0000u),
                                    __uint_as_float(h.y << 16), __uint_as_float(h.y & 0xFFFF0000u)};
        *(RGC_LDS u32x2v_t*)(lds + to[nt] + 256 * kRowChunks * mt) = h;
      }
    if (term) {  // what the terms leave of the targets' entries
#pragma unroll
      for (int mt = 0; mt < MI; ++mt) {
        const int row = 16 * MI * wm + 16 * mt + li, at = rows->at[row] - first;
        if (__any(at >= 0 && at < 16 * NI)) {
#pragma unroll
          for (int nt = 0; nt < NI; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (16 * nt + e == at) a.rest[m0 + row] = t.acc[mt][nt][e];
        }
      }
    }
    __syncthreads();
    uint16_t* out = (term ? a.lo : a.hi) + (m0 + row0) * a.ldd + n0 + 8 * q;
#pragma unroll 4
    for (int it = 0; it < Tile::kRows / kRowsAtOnce; ++it, out += kRowsAtOnce * a.ldd)
      if (m0 + row0 + it * kRowsAtOnce < a.T)
        *reinterpret_cast<u32x4v_t*>(out) = *(const RGC_LDS u32x4v_t*)(lds + 16 * (threadIdx.x + it * kGtThreads));
  }
}

// The logits' kernel of both directions: the tile of this workgroup.
template <bool BACKWARD, bool FEW>
__global__ __launch_bounds__(kGtThreads, FEW ? 4 : 1) void ce_logits_kernel(CeArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[FEW ? FlatTile::kLds : LargeTile::kLds];
  __shared__ CeRows rows;
  int64_t i, j;
  if (!FEW && (int64_t)blockIdx.x < a.grid.large) {
    const int64_t columns = a.grid.split / kGtTile + (a.grid.split % kGtTile != 0);
    gt_place(gt_logical(blockIdx.x, a.grid.large), (a.T + kGtTile - 1) / kGtTile, columns, kCeDown, &i, &j);
    if constexpr (BACKWARD) d_tile<8, 4, 2>(a, i * kGtTile, j * kGtTile, smem, &rows);
    else forward_tile<8, 4, 2>(a, i * kGtTile, j * kGtTile, j, smem, &rows);
    return;
  }
  typedef std::conditional_t<FEW, FlatTile, SmallTile> Tile;
  const int64_t before = a.grid.split / kGtTile;  // columns of large tiles (whole ones where small tiles follow)
  gt_place(gt_logical(blockIdx.x - a.grid.large, gridDim.x - a.grid.large), (a.T + Tile::kRows - 1) / Tile::kRows,
           a.grid.ntiles - before, 2 * kCeDown, &i, &j);
  const int64_t m0 = i * Tile::kRows, n0 = a.grid.split + j * Tile::kCols;
  if constexpr (BACKWARD) {
    if constexpr (FEW) d_tile<2, 2, 3>(a, m0, n0, smem, &rows);
    else d_tile<4, 2, 4>(a, m0, n0, smem, &rows);
  } else {
    if constexpr (FEW) forward_tile<2, 2, 3>(a, m0, n0, before + j, smem, &rows);
    else forward_tile<4, 2, 4>(a, m0, n0, before + j, smem, &rows);
  }
}

template <bool BACKWARD>
__global__ __launch_bounds__(kGtThreads, 4) void ce_pair_kernel(CeArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[PairTile::kLds];
  __shared__ CeRows rows;
  int64_t i, j;
  gt_place(gt_logical(blockIdx.x, gridDim.x), (a.T + PairTile::kRows - 1) / PairTile::kRows, a.grid.ntiles, 2 * kCeDown, &i, &j);
  const int64_t m0 = i * PairTile::kRows, n0 = j * PairTile::kCols;
  if constexpr (BACKWARD) d_tile<4, 2, 2>(a, m0, n0, smem, &rows);
  else forward_tile<4, 2, 2>(a, m0, n0, j, smem, &rows);
}

// C_y += sum of rest_t XP_t over the tokens with target y, in token order. A
// wave per token; the one with a target's first token adds for all of them, eight
// loaded together: one by one they cost a memory latency each. r = 128, 4096 tokens:
// targets drawn evenly from 32768 14 us either way, with frequencies falling as
// 1 / rank 326 us one by one and 89 together, one target for all 3.5 ms and 0.68.
// Each wave looks through the targets for others like its own, so the time grows
// with the tokens' square: 0.42 ms at 32768 even ones, 1.15 at 65536 (16% of a
// call with k = 128).
constexpr int kRestBatch = 8;

__global__ __launch_bounds__(256) void ce_rest_kernel(const int64_t* targets, const float* rest, const uint16_t* XP,
                                                      float* C, int64_t T, int64_t V, int r) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const int64_t y = targets[t];
  if (y < 0 || y >= V) return;
  // 512 targets at a time, so that their loads are in flight together (from
  // clamped places: a load under a condition is waited for before the next)
  for (int64_t j0 = 0; j0 < t; j0 += 512) {
    bool same = false;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int64_t j = j0 + 64 * c + lane, other = targets[j < T ? j : T - 1];
      same |= j < t && other == y;
    }
    if (__any(same)) return;
  }
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  int column[4];  // (clamped: lanes behind the last rank load it too)
#pragma unroll
  for (int q = 0; q < 4; ++q) column[q] = lane + 64 * q < r ? lane + 64 * q : r - 1;
  for (int64_t j0 = t; j0 < T; j0 += 512) {
    uint64_t same[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int64_t j = j0 + 64 * c + lane, other = targets[j < T ? j : T - 1];
      same[c] = __ballot(j < T && other == y);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint64_t m = same[c];
      while (__builtin_popcountll(m) > 2) {
        // up to kRestBatch tokens loaded together (the last again where they are fewer), then added in order
        const int count = __builtin_popcountll(m);
        float w[kRestBatch];
        uint16_t x[kRestBatch][4];
        int at = 0;
#pragma unroll
        for (int b = 0; b < kRestBatch; ++b) {
          if (m) at = __builtin_ctzll(m), m &= m - 1;
          const int64_t j = j0 + 64 * c + at;
          w[b] = rest[j];
#pragma unroll
          for (int q = 0; q < 4; ++q) x[b][q] = XP[j * r + column[q]];
        }
#pragma unroll
        for (int b = 0; b < kRestBatch; ++b)
          if (b < count) {
#pragma unroll
            for (int q = 0; q < 4; ++q) sum[q] = __builtin_fmaf(w[b], bf16_bits_to_f32(x[b][q]), sum[q]);
          }
      }
      while (m) {
        const int64_t j = j0 + 64 * c + __builtin_ctzll(m);
        m &= m - 1;
        const float w = rest[j];
#pragma unroll
        for (int q = 0; q < 4; ++q) sum[q] = __builtin_fmaf(w, bf16_bits_to_f32(XP[j * r + column[q]]), sum[q]);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (lane + 64 * q < r) C[y * r + lane + 64 * q] += sum[q];
}

struct DxArgs {
  const uint16_t* D;  // T x ldd, the piece's hi terms; the lo terms follow
  const uint16_t* W;  // the piece's first row
  int64_t ldd, ldw;
  int64_t T, K, k;    // K: rows of the piece
  int64_t mtiles, ntiles;
  int64_t steps;      // 64-row steps of K to each split
  float* slab;        // [split][T][k] fp32, or null (one piece, one split)
  int first;          // the first piece: the slab is written, not added to
  uint16_t* dX;       // the last piece of an unsplit product: rounded here; else null
  int64_t lddx;
  const uint16_t* V0;  // W's first row
  const int64_t* targets;
  const float* rest;
  int64_t vocab;
};

// rest_t and the row of W it multiplies; 0 and W's first row for an ignored token.
__device__ __forceinline__ float rest_of(const DxArgs& a, int64_t t, const uint16_t** row) {
  const int64_t y = a.targets[t];
  const bool live = y >= 0 && y < a.vocab;
  *row = a.V0 + (live ? y : 0) * a.ldw;
  return live ? a.rest[t] : 0.f;
}

// Tokens of a tile of dX, two rows each (hi and lo). What the second term costs:
// loss and gradient of 4096 x 131072 x 4096 at r = 128 11.5 ms with hi alone, 15.1
// with both; 1001 x 50001 x 2048 frozen 594 and 776 us.
constexpr int kDxTokens = kGtTile / 2;

__global__ __launch_bounds__(kGtThreads, 1) void ce_dx_kernel(DxArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[GtTile<8, 4, 2, true>::kLds];
  const int64_t tiles = a.mtiles * a.ntiles;
  const int64_t place = gt_logical(blockIdx.x, gridDim.x);
  const int64_t split = place / tiles;
  int64_t i, j;
  gt_place(place - split * tiles, a.mtiles, a.ntiles, kCeDown, &i, &j);
  const int64_t m0 = i * kDxTokens, n0 = j * kGtTile;
  const int64_t k0 = split * a.steps * kGtStep;
  const int64_t K = a.K - k0 < a.steps * kGtStep ? a.K - k0 : a.steps * kGtStep;
  GtTile<8, 4, 2, true> t;
  // (hi and lo are 2^28 bytes at most together, so their distance fits a copy's 32-bit offset)
  t.init<true>(a.D + m0 * a.ldd + k0, a.ldd, a.W + k0 * a.ldw + n0, a.ldw, a.T - m0, a.k - n0, K, smem, a.T * a.ldd);
  if (K > 0) t.run();

  const int g = t.lane >> 4, li = t.lane & 15, wm = t.wave & 1, wn = t.wave >> 1;
  float* slab = a.slab ? a.slab + split * a.T * a.k : nullptr;
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    const int64_t row = m0 + 64 * wm + 16 * mt + li;
    if (row >= a.T) continue;
    const uint16_t* wy = nullptr;
    const float rest = a.dX ? rest_of(a, row, &wy) : 0.f;
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const int64_t col = n0 + 64 * wn + 16 * nt + 4 * g;
      if (col >= a.k) continue;  // k is a multiple of 8: four columns are all in or all out
      f32x4_t v = t.acc[mt][nt] + t.acc[mt + 4][nt];
      if (!a.first) v += *reinterpret_cast<const f32x4_t*>(slab + row * a.k + col);
      if (a.dX) {
        if (rest != 0.f) {
          float w[4];
          load_bf16_row<4>(wy + col, w);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(rest, w[e], v[e]);
        }
        *reinterpret_cast<uint2*>(a.dX + row * a.lddx + col) =
            make_uint2(f32x2_to_bf16x2_rne(v[0], v[1]), f32x2_to_bf16x2_rne(v[2], v[3]));
      } else {
        *reinterpret_cast<f32x4_t*>(slab + row * a.k + col) = v;
      }
    }
  }
}

// dX = bf16(sum of the slabs + rest W_y), eight columns to a thread. GROUPS > 1:
// that many threads share the slabs of eight columns (thread group q takes slabs
// q, q + GROUPS, ...) and join through LDS in order of q.
template <int GROUPS>
__global__ __launch_bounds__(256) void ce_join_kernel(DxArgs a, int splits) {
  constexpr int kVectors = 256 / GROUPS;
  __shared__ f32x4_t parts[GROUPS > 1 ? GROUPS : 1][kVectors][2];
  const int v = threadIdx.x % kVectors, q = threadIdx.x / kVectors;
  const int64_t at = ((int64_t)blockIdx.x * kVectors + v) * 8, all = a.T * a.k;
  f32x4_t lo = {0.f, 0.f, 0.f, 0.f}, hi = {0.f, 0.f, 0.f, 0.f};
  if (at < all) {
#pragma unroll 4
    for (int s = q; s < splits; s += GROUPS) {
      lo += *reinterpret_cast<const f32x4_t*>(a.slab + s * all + at);
      hi += *reinterpret_cast<const f32x4_t*>(a.slab + s * all + at + 4);
    }
  }
  if constexpr (GROUPS > 1) {
    parts[q][v][0] = lo;
    parts[q][v][1] = hi;
    __syncthreads();
    if (q > 0) return;
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) {
      lo += parts[i][v][0];
      hi += parts[i][v][1];
    }
  }
  if (at >= all) return;
  const int64_t row = at / a.k, col = at - row * a.k;
  const uint16_t* wy;
  const float rest = rest_of(a, row, &wy);
  if (rest != 0.f) {
    float w[8];
    load_bf16_row<8>(wy + col, w);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo[e] = __builtin_fmaf(rest, w[e], lo[e]);
      hi[e] = __builtin_fmaf(rest, w[e + 4], hi[e]);
    }
  }
  *reinterpret_cast<uint4*>(a.dX + row * a.lddx + col) =
      make_uint4(f32x2_to_bf16x2_rne(lo[0], lo[1]), f32x2_to_bf16x2_rne(lo[2], lo[3]), f32x2_to_bf16x2_rne(hi[0], hi[1]),
                 f32x2_to_bf16x2_rne(hi[2], hi[3]));
}

// XP for the accumulation, `copies` times over (for the two terms of D), with
// zeros for the ignored tokens: D's zeros would not cancel an Inf or NaN there.
// Four values to a thread.
__global__ __launch_bounds__(256) void ce_xp_kernel(const uint2* XP, const int64_t* targets, int64_t V, int64_t T, int quads,
                                                    int copies, uint2* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= T * quads) return;
  const int64_t y = targets[i / quads];
  const uint2 v = y >= 0 && y < V ? XP[i] : make_uint2(0u, 0u);
  for (int c = 0; c < copies; ++c) out[c * T * quads + i] = v;
}

int64_t tiles_of(int64_t n) { return (n + kGtTile - 1) / kGtTile; }
int64_t dx_rows(int64_t T) { return (T + kDxTokens - 1) / kDxTokens; }  // rows of tiles of dX
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Whether the logits take 64-row tiles, and whether one tile holds all tokens.
bool few_tokens(int64_t T) { return T <= FlatTile::kRows; }
bool one_tile(int64_t T) { return T <= SmallTile::kRows; }

// Divides T x V logits into tiles. Large tiles run at the highest rate, but a
// last round of them that fills few compute units costs as much as a full one:
// then the columns of whole rounds stay large and the rest is cut into small
// tiles, which do a quarter of a large one's work at kCeSmallRate of its rate.
// 1001 x 50001 x 2048 (784 large tiles are 3.06 rounds): 221 us with large tiles
// alone, 191 us so; 100 x 12000 x 2048 (47 large tiles): 58 and 28 us.
CeGrid grid_of(int64_t T, int64_t V) {
  const int64_t cus = device_compute_units(), m = tiles_of(T), n = tiles_of(V);
  CeGrid g{};
  if (few_tokens(T)) {
    g.ntiles = (V + FlatTile::kCols - 1) / FlatTile::kCols;
    return g;
  }
  const auto small_columns = [&](int64_t from) { return V > from ? (V - from + SmallTile::kCols - 1) / SmallTile::kCols : 0; };
  const int64_t small_rows = (T + SmallTile::kRows - 1) / SmallTile::kRows;
  const int64_t rounds = m * n / cus;
  double best = (double)((m * n + cus - 1) / cus);
  int64_t columns = n;  // of large tiles
  if (one_tile(T)) best = 1e30, columns = 0;  // half of a large tile's rows would be empty
  for (int64_t keep = one_tile(T) ? 0 : rounds; keep >= 0 && keep >= rounds - 1; --keep) {
    const int64_t c = keep * cus / m < n ? keep * cus / m : n;
    const int64_t small = small_rows * small_columns(c * kGtTile);
    const double cost = (double)((m * c + cus - 1) / cus) + (double)((small + cus - 1) / cus) * 0.25 / kCeSmallRate;
    if (cost < 0.97 * best) best = cost, columns = c;
  }
  g.large = m * columns;
  g.split = columns == n ? V : columns * kGtTile;
  g.ntiles = columns + (columns == n ? 0 : small_columns(g.split));
  return g;
}

// Workgroups of the grid.
int64_t blocks_of(int64_t T, int64_t V, const CeGrid& g) {
  if (few_tokens(T)) return g.ntiles;
  const int64_t before = g.split == V ? g.ntiles : g.split / kGtTile;  // columns of large tiles
  return g.large + (T + SmallTile::kRows - 1) / SmallTile::kRows * (g.ntiles - before);
}

// Whether a launch takes two workgroups to a compute unit, one's epilogue under
// the other's product: where there are no large tiles and more small ones than
// compute units. 300 x 20000 x 1024 (471 tiles): forward 34 us with one workgroup
// on four stages, 26 us so; 300 x 20000 x 4096: 100 and 73 us. Where no unit gets a
// second the deeper stages win, 100 x 12000 x 2048 (94): 29 and 33 us. So they do
// in a forward of several rounds with little epilogue to hide: 128 x 70000 x 4096
// (547) 163 and 189 us, 128 x 95000 x 2048 (743) 111 and 119, but 128 x 70000 x 1024
// 51 and 45; the backwards of the three gain 8, 2 and 12 %. The tile's own sketch
// needs the larger LDS.
bool pair_tiles(const CeArgs& a, int64_t blocks, bool backward) {
  const int64_t cus = device_compute_units();
  return a.grid.large == 0 && !a.C && blocks > cus && (backward || blocks <= 2 * cus || a.k <= 1024);
}

template <bool BACKWARD>
rgc_status_t logits_launch(CeArgs& a, hipStream_t s) {
  a.grid = grid_of(a.T, a.V);
  const int64_t blocks = blocks_of(a.T, a.V, a.grid);
  const dim3 grid((unsigned)blocks), threads(kGtThreads);
  if (few_tokens(a.T)) hipLaunchKernelGGL((ce_logits_kernel<BACKWARD, true>), grid, threads, 0, s, a);
  else if (pair_tiles(a, blocks, BACKWARD)) hipLaunchKernelGGL((ce_pair_kernel<BACKWARD>), grid, threads, 0, s, a);
  else hipLaunchKernelGGL((ce_logits_kernel<BACKWARD, false>), grid, threads, 0, s, a);
  return hipGetLastError() == hipSuccess ? RGC_OK : RGC_ERR_HIP;
}

// How the backward goes through the vocabulary and divides dX's sums.
struct Plan {
  int64_t piece;   // vocabulary rows of a piece
  int64_t pieces;
  int64_t splits;  // of dX's sums within a piece
  bool fused;      // the sketch from the tiles of D themselves
  bool stacked;    // hi and lo in one accumulation of 2 T tokens
  size_t d, xp, rest, slab, acc;  // bytes of the workspace's parts
  size_t total() const { return d + xp + rest + slab + acc; }
};

Plan plan_of(int64_t T, int64_t V, int64_t k, int64_t r) {
  Plan p{};
  p.fused = r > 0 && one_tile(T);
  // a piece's D, two terms, fills the 256 MB last-level cache at most
  int64_t piece = (int64_t(256) << 20) / (T * 4) / kGtTile * kGtTile;
  if (piece < 1024) piece = 1024;
  if (piece > kMaxTiledDim) piece = kMaxTiledDim;
  p.pieces = (V + piece - 1) / piece;
  p.piece = tiles_of((V + p.pieces - 1) / p.pieces) * kGtTile;
  p.pieces = (V + p.piece - 1) / p.piece;
  // as many splits as take the least time: rounds of tiles on the compute units
  // (4.7 TFLOP/s each with all at work), and the slabs' way to memory and back
  // at 4 TB/s. At least four steps to a split.
  const int64_t tiles = dx_rows(T) * tiles_of(k), cus = device_compute_units();
  const int64_t steps = (p.piece + kGtStep - 1) / kGtStep;
  double best = 1e30;
  p.splits = 1;
  for (int64_t s = 1; s <= kCeMaxSplit && (s == 1 || 4 * s <= steps); ++s) {
    const int64_t own = (steps + s - 1) / s;
    const double cost = (double)((tiles * s + cus - 1) / cus) * (double)own * (2.0 * kGtTile * kGtTile * kGtStep / 4.7e12) +
                        (s > 1 ? (double)(s * T * k) * 8 / 4e12 : 0.0);
    if (cost < best) best = cost, p.splits = s;
  }
  p.stacked = 2 * T <= kMaxTiledDim;
  p.d = up256((size_t)(T * p.piece) * 4);
  p.xp = r > 0 && !p.fused ? up256((size_t)((p.stacked ? 2 : 1) * T * r) * 2) : 0;
  p.rest = up256((size_t)T * 4);
  p.slab = p.pieces > 1 || p.splits > 1 ? up256((size_t)(p.splits * T * k) * 4) : 0;
  if (r > 0 && !p.fused) {
    // every width the pieces have: the whole ones and the last
    const int64_t tokens = p.stacked ? 2 * T : T, last = V - (p.pieces - 1) * p.piece;
    const size_t a = rgc_accumulate_workspace_size(tokens, p.piece, r), b = rgc_accumulate_workspace_size(tokens, last, r);
    p.acc = up256(a > b ? a : b);
  }
  return p;
}

rgc_status_t check_rows(const void* p, int64_t ld, int64_t width) {
  if (!p) return RGC_ERR_NULL;
  if (ld < width) return RGC_ERR_SHAPE;
  if (ld > kMaxLeadingDim) return RGC_ERR_UNSUPPORTED;
  if (!aligned16(p) || (ld % 8) != 0) return RGC_ERR_ALIGN;
  return RGC_OK;
}

bool shape_ok(int64_t T, int64_t V, int64_t k, int64_t r) {
  return T > 0 && V > 0 && k > 0 && r >= 0 && r <= k && T <= kMaxTiledDim && V <= kCeMaxVocab && k <= kMaxTiledDim &&
         k % 8 == 0 && (r == 0 || rank_supported(r));
}

rgc_status_t check_shape(int64_t T, int64_t V, int64_t k, int64_t r) {
  if (T < 0 || V <= 0 || k <= 0 || r < 0 || r > k) return RGC_ERR_SHAPE;
  if (T > 0 && !shape_ok(T, V, k, r)) return RGC_ERR_UNSUPPORTED;
  return RGC_OK;
}

rgc_status_t launched() { return hipGetLastError() == hipSuccess ? RGC_OK : RGC_ERR_HIP; }

// Whether the forward's one launch over all tiles stays below 2^31 threads.
bool forward_fits(int64_t T, int64_t V) { return blocks_of(T, V, grid_of(T, V)) < int64_t(1) << 22; }

// A token's partial sums, one for each column of tiles.
size_t part_bytes(int64_t T, int64_t V) { return up256((size_t)grid_of(T, V).ntiles * (size_t)T * 8); }

}  // namespace
}  // namespace rgc

using namespace rgc;

extern "C" size_t rgc_linear_cross_entropy_forward_workspace_size(int64_t T, int64_t V, int64_t k, int64_t r) {
  if (!shape_ok(T, V, k, r) || !forward_fits(T, V)) return 0;
  return part_bytes(T, V) + up256((size_t)T * 4) + (r > 0 ? rgc_project_workspace_size(T, k, r) : 0);
}

extern "C" rgc_status_t rgc_linear_cross_entropy_forward(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
                                                         const uint16_t* P, const int64_t* targets, float* loss,
                                                         float* lse, uint16_t* XP, int64_t T, int64_t V, int64_t k,
                                                         int64_t r, void* ws, size_t ws_bytes, void* stream) {
  rgc_status_t st = check_shape(T, V, k, r);
  if (st != RGC_OK || T == 0) return st;
  if (!forward_fits(T, V)) return RGC_ERR_UNSUPPORTED;
  if ((st = check_rows(X, ldx, k)) != RGC_OK) return st;
  if ((st = check_rows(W, ldw, k)) != RGC_OK) return st;
  if (!targets || !loss || !lse || (r > 0 && (!P || !XP))) return RGC_ERR_NULL;
  if (!aligned_to(targets, 8) || !aligned_to(loss, 4) || !aligned_to(lse, 4) ||
      (r > 0 && (!aligned16(P) || !aligned16(XP))))
    return RGC_ERR_ALIGN;
  if (!ws || ws_bytes < rgc_linear_cross_entropy_forward_workspace_size(T, V, k, r)) return RGC_ERR_WORKSPACE;
  if (!aligned_to(ws, 256)) return RGC_ERR_ALIGN;
  char* at = static_cast<char*>(ws);
  CeArgs a{};
  a.X = X, a.W = W, a.targets = targets, a.ldx = ldx, a.ldw = ldw, a.T = T, a.V = a.vocab = V, a.k = k;
  a.part = reinterpret_cast<float2*>(at);
  at += part_bytes(T, V);
  a.zt = reinterpret_cast<float*>(at);
  at += up256((size_t)T * 4);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (r > 0) {  // the layer's X P, as rgc_project makes it
    st = rgc_project(X, ldx, P, XP, T, k, r, at, ws_bytes - (size_t)(at - static_cast<char*>(ws)), stream);
    if (st != RGC_OK) return st;
  }
  if ((st = logits_launch<false>(a, s)) != RGC_OK) return st;
  hipLaunchKernelGGL(ce_finish_kernel, dim3((unsigned)((T + 15) / 16)), dim3(1024), 0, s, a, loss, lse);
  return launched();
}

extern "C" size_t rgc_linear_cross_entropy_backward_workspace_size(int64_t T, int64_t V, int64_t k, int64_t r) {
  if (!shape_ok(T, V, k, r)) return 0;
  return plan_of(T, V, k, r).total();
}

extern "C" rgc_status_t rgc_linear_cross_entropy_backward(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
                                                          const int64_t* targets, const float* lse, const float* grad,
                                                          const uint16_t* XP, float* C, uint16_t* dX, int64_t lddx,
                                                          int64_t T, int64_t V, int64_t k, int64_t r, void* ws,
                                                          size_t ws_bytes, void* stream) {
  rgc_status_t st = check_shape(T, V, k, r);
  if (st != RGC_OK || T == 0) return st;
  if (r > 0 && V % 8 != 0) return RGC_ERR_UNSUPPORTED;  // the sketch has a layer's widths
  if ((st = check_rows(X, ldx, k)) != RGC_OK) return st;
  if ((st = check_rows(W, ldw, k)) != RGC_OK) return st;
  if ((dX || r == 0) && (st = check_rows(dX, lddx, k)) != RGC_OK) return st;
  if (!targets || !lse || !grad || (r > 0 && (!XP || !C))) return RGC_ERR_NULL;
  if (!aligned_to(targets, 8) || !aligned_to(lse, 4) || !aligned_to(grad, 4) ||
      (r > 0 && (!aligned16(XP) || !aligned16(C))))
    return RGC_ERR_ALIGN;
  const Plan p = plan_of(T, V, k, r);
  if (!ws || ws_bytes < p.total()) return RGC_ERR_WORKSPACE;
  if (!aligned_to(ws, 256)) return RGC_ERR_ALIGN;
  char* at = static_cast<char*>(ws);
  uint16_t* D = reinterpret_cast<uint16_t*>(at);
  uint16_t* xp = reinterpret_cast<uint16_t*>(at + p.d);
  float* slab = p.slab ? reinterpret_cast<float*>(at + p.d + p.xp + p.rest) : nullptr;
  char* acc = at + p.d + p.xp + p.rest + p.slab;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool accumulate = r > 0 && !p.fused;
  if (accumulate) {
    const int64_t n = T * r / 4;
    hipLaunchKernelGGL(ce_xp_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, reinterpret_cast<const uint2*>(XP),
                       targets, V, T, (int)(r / 4), p.stacked ? 2 : 1, reinterpret_cast<uint2*>(xp));
    if ((st = launched()) != RGC_OK) return st;
  }
  CeArgs a{};
  a.X = X, a.targets = targets, a.ldx = ldx, a.ldw = ldw, a.T = T, a.vocab = V, a.k = k;
  a.lse = lse, a.grad = grad;
  a.rest = reinterpret_cast<float*>(at + p.d + p.xp);
  DxArgs x{};
  x.ldw = ldw, x.T = T, x.k = k, x.mtiles = dx_rows(T), x.ntiles = tiles_of(k), x.slab = slab, x.lddx = lddx;
  x.V0 = W, x.targets = targets, x.rest = a.rest, x.vocab = V;
  for (int64_t q = 0; q < p.pieces; ++q) {
    const int64_t v0 = q * p.piece, rows = V - v0 < p.piece ? V - v0 : p.piece;
    a.W = W + v0 * ldw, a.V = rows, a.v0 = v0;
    a.ldd = tiles_of(rows) * kGtTile;
    a.hi = D, a.lo = dX || accumulate ? D + T * a.ldd : nullptr;
    if (p.fused) a.C = C + v0 * r, a.XP = XP, a.r = (int)r;
    if ((st = logits_launch<true>(a, s)) != RGC_OK) return st;
    if (dX) {
      x.D = a.hi, x.W = a.W, x.ldd = a.ldd, x.K = rows, x.first = q == 0;
      x.steps = ((rows + kGtStep - 1) / kGtStep + p.splits - 1) / p.splits;
      x.dX = p.splits == 1 && q == p.pieces - 1 ? dX : nullptr;
      hipLaunchKernelGGL(ce_dx_kernel, dim3((unsigned)(x.mtiles * x.ntiles * p.splits)), dim3(kGtThreads), 0, s, x);
      if ((st = launched()) != RGC_OK) return st;
    }
    if (accumulate) {
      float* c = C + v0 * r;
      if (p.stacked) {
        st = rgc_accumulate(D, a.ldd, xp, c, 2 * T, rows, r, acc, p.acc, stream);
      } else {
        st = rgc_accumulate(a.hi, a.ldd, xp, c, T, rows, r, acc, p.acc, stream);
        if (st == RGC_OK) st = rgc_accumulate(a.lo, a.ldd, xp, c, T, rows, r, acc, p.acc, stream);
      }
      if (st != RGC_OK) return st;
    }
  }
  if (accumulate) {
    hipLaunchKernelGGL(ce_rest_kernel, dim3((unsigned)((T + 3) / 4)), dim3(256), 0, s, targets, a.rest, XP, C, T, V,
                       (int)r);
    if ((st = launched()) != RGC_OK) return st;
  }
  if (dX && p.splits > 1) {
    x.dX = dX;
    const int64_t vectors = T * k / 8;  // (128 slabs of 3 x 512 in 14 us by one thread each)
    if (p.splits >= 32)
      hipLaunchKernelGGL(ce_join_kernel<8>, dim3((unsigned)((vectors + 31) / 32)), dim3(256), 0, s, x, (int)p.splits);
    else
      hipLaunchKernelGGL(ce_join_kernel<1>, dim3((unsigned)((vectors + 255) / 256)), dim3(256), 0, s, x, (int)p.splits);
    st = launched();
  }
  return st;
}
