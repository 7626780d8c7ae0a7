// A tile of A B in bf16 MFMA with fp32 sums, for kernels that do something with
// the products before (or instead of) storing them.
//
// A: M x K with K contiguous. B: N x K with K contiguous (BKM false) or
// K x N with N contiguous (BKM true). Eight waves, two per SIMD, 2 x 4 over
// the tile; a wave makes 16 MI rows by 16 NI columns. MI = 8, NI = 4 is the
// 256 x 256 tile for everything large; 4, 2 (128 x 128) and 2, 2 (64 x 128) fill
// the chip where the large tile leaves compute units idle.
//
// * A step is 64 of K: 128 bytes of a K-contiguous row, a whole cache line
//   (half lines are fetched from L2 twice). Both slabs of a step go straight
//   from memory into one of STAGES LDS stages, STAGES - 1 steps ahead.
// * A wave works in four phases a step, each of MFMAs on a quarter of its block
//   (half its rows x half its columns), and reads the fragments of the next phase
//   from LDS meanwhile: A0 B0 | A0 B1 | A1 B1 | A1 B0. The last phase reads
//   the next step's A0 and B0 into the registers of A0 and B1, which are free
//   by then, so the two B register sets change places every step.
// * One barrier a step, before the last phase: every wave has read all of the
//   step's stage by then, so it is refilled, and the next step's copies have
//   been waited for.
// * LDS rows of 128 bytes: 16-byte chunk q of row t sits at slot q ^ (t % 8),
//   which reads sixteen lanes a clock without a bank conflict (counted: none).
//   With q ^ (t % 8) ^ (t / 8 % 2), which would suit sixteen consecutive
//   lanes, half of the LDS cycles were conflicts. K-major slabs
//   are blocks of 4 K rows x 16 columns read with transposing reads, block
//   (kq, b) at place b ^ (kq / 2 % 2) of its row of sixteen.
// * The MFMA takes B's fragment on its M side, so a lane ends with four
//   consecutive columns of a row: lane (li, g) of wave (wm, wn) holds
//   out[16 MI wm + 16 mt + li][16 NI wn + 16 nt + 4 g + e] in acc[mt][nt][e].
// * Each sum runs over K in ascending order, whatever the launch.
//
// 4096 x 32768 x 4096 on MI355X: MFMAs issue in 93% of the cycles of a short
// run (1.9 PFLOP/s); run after run the card's power holds the clock down to
// 1.2 - 1.3 PFLOP/s, where the library's product of that shape is held too.
#pragma once

#include "rgc_internal.hpp"

namespace rgc {

constexpr int kGtTile = 256;
constexpr int kGtStep = 64;
constexpr int kGtThreads = 512;

struct GtFrag {
  uint32_t r[4];
};

template <int MI, int NI, int STAGES, bool BKM>
struct GtTile {
  static_assert(MI % 2 == 0 && NI % 2 == 0 && (!BKM || NI == 4), "halves; K-major slabs are 256 columns wide");
  static constexpr int kRows = 32 * MI, kCols = 64 * NI;
  static constexpr int kCopiesA = kRows / 64, kCopies = kCopiesA + kCols / 64;  // 1 KB copies of a wave and step
  static constexpr int kSlabA = 128 * kRows, kStage = kSlabA + 128 * kCols;
  static constexpr int kLds = STAGES * kStage;
  static constexpr int MH = MI / 2, NH = NI / 2;

  f32x4_t acc[MI][NI];
  // row and column halves of the fragments, each for the two 32-K halves of a step
  GtFrag a0[MH][2], a1[MH][2], b0[NH][2], b1[NH][2];
  uint32_t voff[kCopies];  // this lane's byte offsets of the wave's copies: A's, then B's (K-major: one)
  uint32_t fa[2], fb[2];
  const uint16_t* A;
  const uint16_t* B;
  int64_t ldb, K, nsteps;
  uint32_t lds0;
  RGC_LDS char* lds;
  int lane, wave;

  // m_rem, n_rem: rows of A and columns of the product that exist (>= 1); what
  // lies behind them is read from the last one and must not be used.
  // PAIRED: the tile takes kRows / 2 rows of A and the same rows of a second matrix
  // `second` elements behind it. A wave's first half of its rows comes from A, the
  // other from the second, so that acc[mt] and acc[mt + MH] belong together.
  template <bool PAIRED = false>
  __device__ __forceinline__ void init(const uint16_t* A_, int64_t lda, const uint16_t* B_, int64_t ldb_, int64_t m_rem,
                                       int64_t n_rem, int64_t K_, char* smem, int64_t second = 0) {
    A = A_, B = B_, ldb = ldb_, K = K_;
    nsteps = (K + kGtStep - 1) / kGtStep;
    lane = threadIdx.x & 63;
    wave = wave_index();
    lds = (RGC_LDS char*)smem;
    lds0 = (uint32_t)(uintptr_t)lds;
    const int g = lane >> 4, li = lane & 15;
#pragma unroll
    for (int v = 0; v < kCopies; ++v) {
      const bool of_a = v < kCopiesA;
      const int c = wave + 8 * (of_a ? v : v - kCopiesA);  // 1 KB of the slab
      if (of_a || !BKM) {
        // eight rows of 128 bytes; lane l fills slot l % 8 of row l / 8
        const int64_t last = (of_a ? m_rem : n_rem) - 1;
        int64_t row = 8 * c + (lane >> 3), from = 0;
        if (PAIRED && of_a) {
          const int in_wave = (int)row % (16 * MI);
          from = in_wave >= 16 * MH ? second : 0;
          row = 16 * MH * (row / (16 * MI)) + in_wave % (16 * MH);
        }
        row = row < last ? row : last;
        voff[v] = (uint32_t)((from + row * (of_a ? lda : ldb) + 8 * chunk()) * 2);
      } else if (v == kCopiesA) {
        int64_t col = column(c);
        col = col + 8 <= n_rem ? col : n_rem - 8;
        voff[v] = (uint32_t)((krow(c) * ldb + col) * 2);
      }
    }
    const int swz = li & 7;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      fa[kk] = (uint32_t)(128 * (16 * MI * (wave & 1) + li) + 16 * ((4 * kk + g) ^ swz));
      if constexpr (!BKM) fb[kk] = (uint32_t)(kSlabA + 128 * (16 * NI * (wave >> 1) + li) + 16 * ((4 * kk + g) ^ swz));
    }
    if constexpr (BKM) {
      // block rows kq = 8 kk + 2 g + h: kq / 2 % 2 = g % 2, so even and odd blocks change places where g is odd
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
        fb[nt] = (uint32_t)(kSlabA + 128 * (32 * g + 4 * (wave >> 1) + (nt ^ (g & 1))) + 8 * li);
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }

  // chunk of its row that a lane fetches (K-contiguous slabs)
  __device__ __forceinline__ int chunk() const { return (lane & 7) ^ (lane >> 3); }
  // K row and column that lane l of copy c fetches (K-major slabs): blocks 8 c .. 8 c + 7
  __device__ __forceinline__ int krow(int c) const { return 4 * (c >> 1) + ((lane & 7) >> 1); }
  __device__ __forceinline__ int64_t column(int c) const {
    const int place = 8 * (c & 1) + (lane >> 3);
    return 16 * (place ^ ((c >> 2) & 1)) + 8 * (lane & 1);
  }

  // Copy v of this wave, from the step's bases. `left`: elements of K from the
  // step on; where they are fewer than a step, the lanes behind the end fetch
  // the last chunk (or K row) instead, which settle() clears or A's zeros cancel.
  __device__ __forceinline__ void copy(int v, const uint16_t* Ab, const uint16_t* Bb, uint32_t st, int left) const {
    const bool of_a = v < kCopiesA;
    const int c = wave + 8 * (of_a ? v : v - kCopiesA);
    if (of_a || !BKM) {
      const int over = chunk() - (left - 1) / 8;
      dma_16b_cached(of_a ? Ab : Bb, voff[v] - (uint32_t)(16 * (over > 0 ? over : 0)), st + (of_a ? 0 : kSlabA) + 1024 * c);
    } else {
      // a K-major slab's copies are sixteen K rows apart, so one offset (of a
      // row from 0 to 15) serves the four; base and lane are clamped to the
      // last row each, and the offset never falls below the base
      const int last = left - 1, row0 = 16 * (v - kCopiesA) < last ? 16 * (v - kCopiesA) : last;
      const int over = krow(wave) - (last - row0);
      dma_16b_cached(Bb + row0 * ldb, voff[kCopiesA] - (uint32_t)(over > 0 ? over : 0) * (uint32_t)(2 * ldb),
                     st + kSlabA + 1024 * c);
    }
  }
  __device__ __forceinline__ int left_of(int64_t step) const {
    const int64_t left = K - step * kGtStep;
    return left < kGtStep ? (int)left : kGtStep;
  }
  // stage: a stage's byte offset
  __device__ __forceinline__ void issue(int64_t step, uint32_t stage) const {
    const int64_t k0 = step * kGtStep;
    const uint16_t* Ab = uniform_ptr(A + k0);
    const uint16_t* Bb = uniform_ptr(BKM ? B + k0 * ldb : B + k0);
#pragma unroll
    for (int v = 0; v < kCopies; ++v) copy(v, Ab, Bb, lds0 + stage, left_of(step));
  }
  // After the barrier that ends a step's copies: clears the chunks behind the
  // end of K in the last step.
  __device__ __forceinline__ void settle(int64_t step, uint32_t stage) const {
    const int64_t left = K - step * kGtStep;
    if (left >= kGtStep) return;
    for (int p = threadIdx.x; p < (BKM ? kSlabA : kStage) / 16; p += kGtThreads) {
      const int row = p >> 3, q = (p & 7) ^ (row & 7);  // (both slabs hold a multiple of 8 rows)
      if (8 * q >= left) *(RGC_LDS u32x4v_t*)(lds + stage + 16 * p) = u32x4v_t{0u, 0u, 0u, 0u};
    }
    lds_barrier();
  }

  __device__ __forceinline__ GtFrag read16(uint32_t off) const {
    const u32x4v_t v = *(const RGC_LDS u32x4v_t*)(lds + off);
    return GtFrag{{v.x, v.y, v.z, v.w}};
  }
  template <int H>
  __device__ __forceinline__ void read_a(GtFrag (&a)[MH][2], uint32_t stage) const {
#pragma unroll
    for (int mt = 0; mt < MH; ++mt)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) a[mt][kk] = read16(fa[kk] + stage + 2048 * (MH * H + mt));
  }
  template <int H>
  __device__ __forceinline__ void read_b(GtFrag (&b)[NH][2], uint32_t stage) const {
#pragma unroll
    for (int nt = 0; nt < NH; ++nt)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        if constexpr (BKM) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x2v_t v = lds_read_tr16(lds + fb[nt] + stage + 2048 * (8 * kk + h) + 256 * H);
            b[nt][kk].r[2 * h] = v.x;
            b[nt][kk].r[2 * h + 1] = v.y;
          }
        } else {
          b[nt][kk] = read16(fb[kk] + stage + 2048 * (NH * H + nt));
        }
      }
  }
  template <int HA, int HB>
  __device__ __forceinline__ void multiply(const GtFrag (&a)[MH][2], const GtFrag (&b)[NH][2]) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int mt = 0; mt < MH; ++mt)
#pragma unroll
        for (int nt = 0; nt < NH; ++nt)
          acc[MH * HA + mt][NH * HB + nt] = mfma_16x16x32(b[nt][kk].r, a[mt][kk].r, acc[MH * HA + mt][NH * HB + nt]);
  }

  __device__ __forceinline__ void step(int64_t s, uint32_t stage, uint32_t next, GtFrag (&x)[NH][2], GtFrag (&y)[NH][2]) {
    read_b<1>(y, stage);
    multiply<0, 0>(a0, x);
    __builtin_amdgcn_sched_barrier(0);
    read_a<1>(a1, stage);
    multiply<0, 1>(a0, y);
    __builtin_amdgcn_sched_barrier(0);
    multiply<1, 1>(a1, y);
    __builtin_amdgcn_sched_barrier(0);
    if (s + 1 < nsteps) {
      if (STAGES > 2 && s + STAGES <= nsteps) wait_vmcnt<(STAGES - 2) * kCopies>();
      else wait_vmcnt<0>();
      lds_barrier();
      settle(s + 1, next);
      read_a<0>(a0, next);
      read_b<0>(y, next);
    }
    __builtin_amdgcn_s_setprio(1);
    if (s + STAGES < nsteps) issue(s + STAGES, stage);
    multiply<1, 0>(a1, x);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  }

  // The whole product; ends with a barrier, after which the LDS is free.
  __device__ __forceinline__ void run() {
    const int64_t ahead = nsteps < STAGES ? nsteps : STAGES;
#pragma unroll
    for (int s = 0; s < STAGES; ++s)
      if (s < ahead) issue(s, s * kStage);
    if (ahead == STAGES) wait_vmcnt<(STAGES - 1) * kCopies>();
    else wait_vmcnt<0>();
    lds_barrier();
    settle(0, 0);
    read_a<0>(a0, 0);
    read_b<0>(b0, 0);
    uint32_t stage = 0;
    const auto after = [](uint32_t st) { return st == (STAGES - 1) * kStage ? 0u : st + kStage; };
    for (int64_t s = 0; s < nsteps; s += 2) {
      const uint32_t second = STAGES == 2 ? kStage : after(stage), third = STAGES == 2 ? 0 : after(second);
      step(s, STAGES == 2 ? 0 : stage, second, b0, b1);
      if (s + 1 < nsteps) step(s + 1, second, third, b1, b0);
      stage = third;
    }
    lds_barrier();
  }
};

// The hardware hands workgroups to the XCDs round-robin; this numbers them so
// that each XCD gets a contiguous run.
__device__ __forceinline__ int64_t gt_logical(int64_t b, int64_t G) {
  const int64_t x = b % 8, pos = b / 8, q = G / 8, rem = G % 8;
  return x * q + (x < rem ? x : rem) + pos;
}

// Tile (i, j) of place t in groups of `down` tile rows, each walked down its
// columns, so that the tiles running on one XCD share rows of A and of B.
__device__ __forceinline__ void gt_place(int64_t t, int64_t mtiles, int64_t ntiles, int64_t down, int64_t* i, int64_t* j) {
  const int64_t grp = t / (down * ntiles), within = t - grp * down * ntiles;
  const int64_t rows = mtiles - grp * down < down ? mtiles - grp * down : down;
  *j = within / rows;
  *i = grp * down + within % rows;
}

}  // namespace rgc
