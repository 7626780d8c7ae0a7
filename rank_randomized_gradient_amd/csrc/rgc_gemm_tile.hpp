// One 256 x 256 tile of A B in bf16 MFMA with fp32 sums, for kernels that do
// something with the products before (or instead of) storing them.
//
// A: M x K with K contiguous. B: N x K with K contiguous (BKM false) or
// K x N with N contiguous (BKM true). Eight waves, two per SIMD, 2 x 4 over
// the tile: wave (wm, wn) makes rows 128 wm .. +127 of columns 64 wn .. +63.
//
// * A step is 64 of K: 128 bytes of a K-contiguous row, a whole cache line
//   (half lines are fetched from L2 twice). Both slabs of a step (32 KB each)
//   go straight from memory into one of two LDS stages.
// * A wave works in four phases a step, each sixteen MFMAs on a quarter of its
//   block (64 rows x 32 columns), and reads the fragments of the next phase
//   from LDS meanwhile: A0 B0 | A0 B1 | A1 B1 | A1 B0. The last phase reads
//   the next step's A0 and B0 into the registers of A0 and B1, which are free
//   by then, so the two B register sets change places every step.
// * One barrier a step, before the last phase: every wave has read all of the
//   step's stage by then, so it is refilled for the step after next, and the
//   next step's copies, issued a step ago, have been waited for.
// * LDS rows of 128 bytes: 16-byte chunk q of row t sits at slot q ^ (t % 8),
//   which reads sixteen lanes a clock without a bank conflict (counted: none).
//   With q ^ (t % 8) ^ (t / 8 % 2), which would suit sixteen consecutive
//   lanes, half of the LDS cycles were conflicts. K-major slabs
//   are blocks of 4 K rows x 16 columns read with transposing reads, block
//   (kq, b) at place b ^ (kq / 2 % 2) of its row of sixteen.
// * The MFMA takes B's fragment on its M side, so a lane ends with four
//   consecutive columns of a row: lane (li, g) holds
//   out[128 wm + 16 mt + li][64 wn + 16 nt + 4 g + e] in acc[mt][nt][e].
// * Each sum runs over K in ascending order, whatever the launch.
#pragma once

#include "rgc_internal.hpp"

namespace rgc {

constexpr int kGtTile = 256;
constexpr int kGtStep = 64;
constexpr int kGtThreads = 512;
constexpr int kGtSlab = 32768;
constexpr int kGtStage = 2 * kGtSlab;
constexpr int kGtLds = 2 * kGtStage;

struct GtFrag {
  uint32_t r[4];
};

template <bool BKM>
struct GtTile {
  f32x4_t acc[8][4];
  // 64-row and 32-column halves of the fragments, each for the two 32-K halves of a step
  GtFrag a0[4][2], a1[4][2], b0[2][2], b1[2][2];
  uint32_t voff[8];  // this lane's byte offsets of the wave's copies: four of A, four of B (K-major: one)
  uint32_t fa[2], fb[2];
  const uint16_t* A;
  const uint16_t* B;
  int64_t ldb, K, nsteps;
  uint32_t lds0;
  RGC_LDS char* lds;
  int lane, wave;

  // m_rem, n_rem: rows of A and columns of the product that exist (>= 1); what
  // lies behind them is read from the last one and must not be used.
  __device__ __forceinline__ void init(const uint16_t* A_, int64_t lda, const uint16_t* B_, int64_t ldb_, int64_t m_rem,
                                       int64_t n_rem, int64_t K_, char* smem) {
    A = A_, B = B_, ldb = ldb_, K = K_;
    nsteps = (K + kGtStep - 1) / kGtStep;
    lane = threadIdx.x & 63;
    wave = wave_index();
    lds = (RGC_LDS char*)smem;
    lds0 = (uint32_t)(uintptr_t)lds;
    const int g = lane >> 4, li = lane & 15;
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const int c = wave + 8 * (v & 3);  // 1 KB of the slab
      if (v < 4 || !BKM) {
        // eight rows of 128 bytes; lane l fills slot l % 8 of row l / 8
        const int64_t last = (v < 4 ? m_rem : n_rem) - 1;
        int64_t row = 8 * c + (lane >> 3);
        row = row < last ? row : last;
        voff[v] = (uint32_t)((row * (v < 4 ? lda : ldb) + 8 * chunk()) * 2);
      } else if (v == 4) {
        int64_t col = column(c);
        col = col + 8 <= n_rem ? col : n_rem - 8;
        voff[v] = (uint32_t)((krow(c) * ldb + col) * 2);
      }
    }
    const int swz = li & 7;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      fa[kk] = (uint32_t)(128 * (128 * (wave & 1) + li) + 16 * ((4 * kk + g) ^ swz));
      if constexpr (!BKM) fb[kk] = (uint32_t)(kGtSlab + 128 * (64 * (wave >> 1) + li) + 16 * ((4 * kk + g) ^ swz));
    }
    if constexpr (BKM) {
      // block rows kq = 8 kk + 2 g + h: kq / 2 % 2 = g % 2, so even and odd blocks change places where g is odd
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
        fb[nt] = (uint32_t)(kGtSlab + 128 * (32 * g + 4 * (wave >> 1) + (nt ^ (g & 1))) + 8 * li);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
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
    const int c = wave + 8 * (v & 3);
    if (v < 4 || !BKM) {
      const int over = chunk() - (left - 1) / 8;
      dma_16b_cached(v < 4 ? Ab : Bb, voff[v] - (uint32_t)(16 * (over > 0 ? over : 0)),
                     st + (v < 4 ? 0 : kGtSlab) + 1024 * c);
    } else {
      // a K-major slab's copies are sixteen K rows apart, so one offset (of a
      // row from 0 to 15) serves the four; base and lane are clamped to the
      // last row each, and the offset never falls below the base
      const int last = left - 1, row0 = 16 * (v - 4) < last ? 16 * (v - 4) : last;
      const int over = krow(wave) - (last - row0);
      dma_16b_cached(Bb + row0 * ldb, voff[4] - (uint32_t)(over > 0 ? over : 0) * (uint32_t)(2 * ldb),
                     st + kGtSlab + 1024 * c);
    }
  }
  __device__ __forceinline__ int left_of(int64_t step) const {
    const int64_t left = K - step * kGtStep;
    return left < kGtStep ? (int)left : kGtStep;
  }
  __device__ __forceinline__ void issue(int64_t step, uint32_t stage) const {
    const int64_t k0 = step * kGtStep;
    const uint16_t* Ab = uniform_ptr(A + k0);
    const uint16_t* Bb = uniform_ptr(BKM ? B + k0 * ldb : B + k0);
#pragma unroll
    for (int v = 0; v < 8; ++v) copy(v, Ab, Bb, lds0 + stage * kGtStage, left_of(step));
  }
  // After the barrier that ends a step's copies: clears the chunks behind the
  // end of K in the last step.
  __device__ __forceinline__ void settle(int64_t step, uint32_t stage) const {
    const int64_t left = K - step * kGtStep;
    if (left >= kGtStep) return;
    for (int p = threadIdx.x; p < (BKM ? 1 : 2) * kGtSlab / 16; p += kGtThreads) {
      const int row = (p >> 3) & 255, q = (p & 7) ^ (row & 7);
      if (8 * q >= left) *(RGC_LDS u32x4v_t*)(lds + stage * kGtStage + 16 * p) = u32x4v_t{0u, 0u, 0u, 0u};
    }
    lds_barrier();
  }

  __device__ __forceinline__ GtFrag read16(uint32_t off) const {
    const u32x4v_t v = *(const RGC_LDS u32x4v_t*)(lds + off);
    return GtFrag{{v.x, v.y, v.z, v.w}};
  }
  template <int H>
  __device__ __forceinline__ void read_a(GtFrag (&a)[4][2], uint32_t stage) const {
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) a[mt][kk] = read16(fa[kk] + stage * kGtStage + 8192 * H + 2048 * mt);
  }
  template <int H>
  __device__ __forceinline__ void read_b(GtFrag (&b)[2][2], uint32_t stage) const {
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        if constexpr (BKM) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x2v_t v = lds_read_tr16(lds + fb[nt] + stage * kGtStage + 2048 * (8 * kk + h) + 256 * H);
            b[nt][kk].r[2 * h] = v.x;
            b[nt][kk].r[2 * h + 1] = v.y;
          }
        } else {
          b[nt][kk] = read16(fb[kk] + stage * kGtStage + 4096 * H + 2048 * nt);
        }
      }
  }
  template <int HA, int HB>
  __device__ __forceinline__ void multiply(const GtFrag (&a)[4][2], const GtFrag (&b)[2][2]) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
          acc[4 * HA + mt][2 * HB + nt] = mfma_16x16x32(b[nt][kk].r, a[mt][kk].r, acc[4 * HA + mt][2 * HB + nt]);
  }

  template <int STAGE>
  __device__ __forceinline__ void step(int64_t s, GtFrag (&x)[2][2], GtFrag (&y)[2][2]) {
    read_b<1>(y, STAGE);
    multiply<0, 0>(a0, x);
    __builtin_amdgcn_sched_barrier(0);
    read_a<1>(a1, STAGE);
    multiply<0, 1>(a0, y);
    __builtin_amdgcn_sched_barrier(0);
    multiply<1, 1>(a1, y);
    __builtin_amdgcn_sched_barrier(0);
    if (s + 1 < nsteps) {
      wait_vmcnt<0>();
      lds_barrier();
      settle(s + 1, STAGE ^ 1);
      read_a<0>(a0, STAGE ^ 1);
      read_b<0>(y, STAGE ^ 1);
    }
    __builtin_amdgcn_s_setprio(1);
    if (s + 2 < nsteps) issue(s + 2, STAGE);
    multiply<1, 0>(a1, x);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  }

  // The whole product; ends with a barrier, after which the LDS is free.
  __device__ __forceinline__ void run() {
    issue(0, 0);
    if (nsteps > 1) {
      issue(1, 1);
      wait_vmcnt<8>();
    } else {
      wait_vmcnt<0>();
    }
    lds_barrier();
    settle(0, 0);
    read_a<0>(a0, 0);
    read_b<0>(b0, 0);
    for (int64_t s = 0; s < nsteps; s += 2) {
      step<0>(s, b0, b1);
      if (s + 1 < nsteps) step<1>(s + 1, b1, b0);
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
