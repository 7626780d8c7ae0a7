// Layer norm and root-mean-square norm, forward and backward with the weights'
// gradients, for rows of up to 65536 elements in bf16 or fp32.
//
//   mu = mean(x) (0 for rms), rstd = 1 / sqrt(mean((x - mu)^2) + eps)
//   xhat = (x - mu) rstd,     y = xhat w + b
//   h = dy w,  dx = rstd (h - mean(h) - xhat mean(h xhat))   (rms: without mean(h))
//   dw = sum over rows of dy xhat,   db = sum over rows of dy
//
// Everything is held in fp32; y and dx are rounded once to X's type, dw and db
// once to the weight's type. All four are bound by memory: the forward reads
// x and writes y, the backward reads dy and x and writes dx.
//
// * A row is held in the registers of TPR threads (16 lanes up to a whole
//   workgroup), NV vectors of 8 elements each, so x (and dy) come from
//   memory once: mean, centred squares and the output all use the held values.
// * Vectors are loaded and stored at whatever address the row starts: global
//   memory accesses need no alignment on this part. Only the last vector of a row
//   whose width is no multiple of 8 (RAGGED) goes element by element. (Element
//   by element throughout, rows of 1003 moved at 1.8 TB/s, against 5 TB/s.)
// * Backward: a workgroup walks the rows with a stride of the grid, every thread
//   adding its columns' dy xhat and dy in registers. At the end the
//   workgroup's row groups are added through LDS and one partial row per
//   workgroup goes to the workspace; a second launch adds the partials. The
//   grid is one workgroup per compute unit, which keeps the partials small
//   beside the rows (8 MB beside 100 at 4096 x 4096). Up to 4096 bf16 or
//   2048 fp32 elements a row is one wave's, so no barrier ties the rows in flight to each other. All
//   sums have a fixed order.
// * Backward rows above 16384 elements do not fit the registers: one launch
//   makes the column sums, another dx, reading each row twice (the second time
//   from cache), both element by element: 4096 x 32768 bf16 in 503 us, 1.6 TB/s
//   of x, dy and dx once. (Up to 16384: 8192 x 16384 in 185 us, 4.3 TB/s.)
//
// Measured on MI355X, bf16, where a copy reaches 5.2 TB/s: forward of 32768 x
// 4096 in 104 us (5.1 TB/s), backward in 170 (4.7); 4096 x 4096 in 15 and 32.
// With 1024 threads on four rows at a time and barriers for their sums the
// backward took 430 us. Non-temporal stores saved 5% here and cost the next
// reader of y as much.
#include "rgc_internal.hpp"

namespace rgc {
namespace {

constexpr int64_t kNormMaxWidth = 65536;
constexpr int64_t kNormMaxRows = int64_t(1) << 31;
constexpr int64_t kNormHeldBackward = 16384;  // widest backward row held in registers
constexpr int kBwdThreads = 1024;           // of the wide rows' dx launch
constexpr int kPanel = 256;  // columns of a workgroup of the column-sum launch

struct NormArgs {
  const void* x;
  const void* dy;   // backward
  const void* w;    // null: ones
  const void* b;    // null: none (forward)
  void* out;        // y or dx
  float* mean;      // forward: written unless null; backward: read (layer)
  float* rstd;
  float* part;      // backward: partial rows
  int64_t ldx, lddy, ldo;
  int64_t rows, n;
  float eps;
  int w_f32;
  int centre;
  int db;           // backward: db wanted
};

// Eight elements of a row as loaded, and their values. again() hides from the
// compiler that the values are those of before, so that it unpacks them anew
// instead of keeping them in registers in between.
template <typename XT>
struct Raw;
template <>
struct Raw<uint16_t> {
  typedef u32x4v_t any_t __attribute__((aligned(2)));
  u32x4v_t v;
  __device__ __forceinline__ void zero() { v = u32x4v_t{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void again() { asm volatile("" : "+v"(v)); }
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const any_t*>(p); }
  __device__ __forceinline__ void load_some(const uint16_t* p, int count) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < count) v[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
  }
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16); }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&f)[8]) {
    *reinterpret_cast<any_t*>(p) = u32x4v_t{f32x2_to_bf16x2_rne(f[0], f[1]), f32x2_to_bf16x2_rne(f[2], f[3]),
                                            f32x2_to_bf16x2_rne(f[4], f[5]), f32x2_to_bf16x2_rne(f[6], f[7])};
  }
  static __device__ __forceinline__ void store_some(uint16_t* p, const float (&f)[8], int count) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < count) p[i] = (uint16_t)f32_to_bf16_rne(f[i]);
  }
};
template <>
struct Raw<float> {
  typedef f32x4_t any_t __attribute__((aligned(4)));
  f32x4_t a, b;
  __device__ __forceinline__ void zero() { a = b = f32x4_t{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ void again() {}
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const any_t*>(p)[0];
    b = reinterpret_cast<const any_t*>(p)[1];
  }
  __device__ __forceinline__ void load_some(const float* p, int count) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < count) (i < 4 ? a : b)[i & 3] = p[i];
  }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i & 3] : b[i & 3]; }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
    reinterpret_cast<any_t*>(p)[0] = f32x4_t{f[0], f[1], f[2], f[3]};
    reinterpret_cast<any_t*>(p)[1] = f32x4_t{f[4], f[5], f[6], f[7]};
  }
  static __device__ __forceinline__ void store_some(float* p, const float (&f)[8], int count) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < count) p[i] = f[i];
  }
};

// The vector at column c of a row of n elements: zeros behind the end.
template <bool RAGGED, typename XT>
__device__ __forceinline__ void load_at(Raw<XT>& r, const XT* row, int c, int n) {
  r.zero();
  if (c + 8 <= n) r.load(row + c);
  else if (RAGGED && c < n) r.load_some(row + c, n - c);
}
template <bool RAGGED, typename XT>
__device__ __forceinline__ void store_at(XT* row, int c, int n, const float (&f)[8]) {
  if (c + 8 <= n) Raw<XT>::store(row + c, f);
  else if (RAGGED && c < n) Raw<XT>::store_some(row + c, f, n - c);
}

__device__ __forceinline__ float load_param(const void* p, int f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}
template <bool RAGGED>
__device__ __forceinline__ void load_params(const void* p, int f32, int c, int n, float (&out)[8]) {
  if (f32) {
    Raw<float> r;
    load_at<RAGGED>(r, static_cast<const float*>(p), c, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = r.get(e);
  } else {
    Raw<uint16_t> r;
    load_at<RAGGED>(r, static_cast<const uint16_t*>(p), c, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = r.get(e);
  }
}

// v plus its value R lanes further round a row of sixteen. Every step of a
// halving sequence pairs the same two partial sums in both lanes.
template <int R>
__device__ __forceinline__ float add_rotated(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + R, 0xF, 0xF, false));
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  static_assert(LANES == 16 || LANES == 64, "row or wave");
  v = add_rotated<1>(add_rotated<2>(add_rotated<4>(add_rotated<8>(v))));
  if constexpr (LANES == 64) {
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
  }
  return v;
}

// Sums of N values over the TPR threads of a row group, in all of them: within
// a wave across lanes, across the waves of a wider group through LDS, `slots`
// being N floats per wave of the workgroup, used by one call between two
// barriers (the caller alternates two sets).
template <int TPR, int N>
__device__ __forceinline__ void group_sum(float (&a)[N], float* slots) {
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = lanes_sum<(TPR < 64 ? 16 : 64)>(a[i]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) slots[N * wave + i] = a[i];
    }
    __syncthreads();
    const int w0 = wave / W * W;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      a[i] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) a[i] += slots[N * (w0 + w) + i];
    }
  }
}

// Forward: a workgroup of THREADS threads takes THREADS / TPR rows at a time.
template <typename XT, bool RAGGED, int NV, int TPR, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_forward_kernel(NormArgs a) {
  constexpr int GROUPS = THREADS / TPR;
  __shared__ float slots[2][THREADS / 64];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR, n = (int)a.n;
  const float inv_n = 1.0f / (float)n;
  for (int64_t row0 = (int64_t)blockIdx.x * GROUPS; row0 < a.rows; row0 += (int64_t)gridDim.x * GROUPS) {
    const int64_t row = row0 + grp;
    const bool live = row < a.rows;
    const XT* x = static_cast<const XT*>(a.x) + (live ? row : row0) * a.ldx;
    Raw<XT> raw[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_at<RAGGED>(raw[j], x, (j * TPR + t) * 8, n);
    float mu = 0.f;
    if (a.centre) {
      float s[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += raw[j].get(e);
      group_sum<TPR>(s, slots[0]);
      mu = s[0] * inv_n;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + t) * 8;
      raw[j].again();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = c + (RAGGED ? e : 0) < n ? raw[j].get(e) - mu : 0.f;
        q[0] = __builtin_fmaf(d, d, q[0]);
      }
    }
    group_sum<TPR>(q, slots[1]);
    const float rstd = 1.0f / sqrtf(q[0] * inv_n + a.eps);
    if (live && t == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = rstd;
    }
    XT* y = static_cast<XT*>(a.out) + row * a.ldo;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + t) * 8;
      if (c >= n || !live) continue;
      raw[j].again();
      float f[8], p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = (raw[j].get(e) - mu) * rstd;
      if (a.w) {
        load_params<RAGGED>(a.w, a.w_f32, c, n, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] * p[e];
      }
      if (a.b) {
        load_params<RAGGED>(a.b, a.w_f32, c, n, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] + p[e];
      }
      store_at<RAGGED>(y, c, n, f);
    }
    if constexpr (TPR > 64) __syncthreads();  // before the next rows' sums reuse the slots
  }
}

// Backward with the row in registers; see the head of the file. The weight is
// kept in LDS. With c = x - mu: dw += (g rstd) c, and dx = rstd h - rstd c1 -
// c (rstd^2 c2), c1 = mean(h) and c2 = mean(h c).
template <typename XT, bool RAGGED, int NV, int TPR, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_backward_kernel(NormArgs a) {
  constexpr int GROUPS = THREADS / TPR, COLS = TPR * NV * 8;
  __shared__ float slots[2][2 * THREADS / 64];
  __shared__ __attribute__((aligned(16))) float mem[GROUPS * COLS];  // the weight; at the end the groups' sums
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR, n = (int)a.n;
  const float inv_n = 1.0f / (float)n;
  for (int c = threadIdx.x; c < COLS; c += THREADS)
    mem[c] = c >= n ? 0.f : a.w ? load_param(a.w, a.w_f32, c) : 1.f;
  float dw[NV][8], db[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[j][e] = 0.f, db[j][e] = 0.f;
  __syncthreads();
  const int64_t stride = (int64_t)gridDim.x * GROUPS;
  int parity = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * GROUPS; row0 < a.rows; row0 += stride, parity ^= 1) {
    const int64_t row = row0 + grp;
    const bool live = row < a.rows;
    if (TPR <= 64 && !live) break;  // (wider groups meet at the barriers)
    Raw<XT> rx[NV], rg[NV];
    const XT* x = static_cast<const XT*>(a.x) + (live ? row : 0) * a.ldx;
    const XT* g = static_cast<const XT*>(a.dy) + (live ? row : 0) * a.lddy;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = live ? (j * TPR + t) * 8 : n;
      load_at<RAGGED>(rx[j], x, c, n);
      load_at<RAGGED>(rg[j], g, c, n);
    }
    const float mu = live && a.centre ? a.mean[row] : 0.f, rstd = live ? a.rstd[row] : 0.f;
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float* w = mem + (j * TPR + t) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // columns behind the row's end have g = 0
        const float gv = rg[j].get(e), c = rx[j].get(e) - mu, h = gv * w[e];
        sum[0] += h;
        sum[1] = __builtin_fmaf(h, c, sum[1]);
        dw[j][e] = __builtin_fmaf(gv * rstd, c, dw[j][e]);
        db[j][e] += gv;
      }
      // the sums here and not behind the stores, where the compiler would take them with all they need
#pragma unroll
      for (int e = 0; e < 8; ++e) asm volatile("" : "+v"(dw[j][e]), "+v"(db[j][e]));
    }
    group_sum<TPR>(sum, slots[parity]);
    const float k1 = a.centre ? sum[0] * inv_n * rstd : 0.f, k2 = sum[1] * inv_n * rstd * rstd * rstd;
    XT* dx = static_cast<XT*>(a.out) + row * a.ldo;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + t) * 8;
      if (c >= n || !live) continue;
      rx[j].again();
      rg[j].again();
      const float* w = mem + c;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        f[e] = __builtin_fmaf(rg[j].get(e) * w[e], rstd, -__builtin_fmaf(rx[j].get(e) - mu, k2, k1));
      store_at<RAGGED>(dx, c, n, f);
    }
  }
  // the workgroup's partial rows: dw, then db
  for (int which = 0; which < 1 + a.db; ++which) {
    float* part = a.part + ((int64_t)which * gridDim.x + blockIdx.x) * a.n;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) mem[grp * COLS + (j * TPR + t) * 8 + e] = which ? db[j][e] : dw[j][e];
    __syncthreads();
    for (int64_t c = threadIdx.x; c < n; c += THREADS) {
      float s = 0.f;
#pragma unroll 4
      for (int q = 0; q < GROUPS; ++q) s += mem[q * COLS + c];
      part[c] = s;
    }
  }
}

// Wide rows, second launch: dx, one row per workgroup, each row read twice.
template <typename XT>
__global__ __launch_bounds__(kBwdThreads) void norm_wide_dx_kernel(NormArgs a) {
  __shared__ float slots[2 * kBwdThreads / 64];
  const float inv_n = 1.0f / (float)a.n;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const XT* x = static_cast<const XT*>(a.x) + row * a.ldx;
    const XT* g = static_cast<const XT*>(a.dy) + row * a.lddy;
    XT* dx = static_cast<XT*>(a.out) + row * a.ldo;
    const float mu = a.centre ? a.mean[row] : 0.f, rstd = a.rstd[row];
    float sum[2] = {0.f, 0.f};
    for (int64_t c = threadIdx.x; c < a.n; c += kBwdThreads) {
      const float xv = load_param(x, sizeof(XT) == 4, c), gv = load_param(g, sizeof(XT) == 4, c);
      const float h = gv * (a.w ? load_param(a.w, a.w_f32, c) : 1.f);
      sum[0] += h;
      sum[1] += h * ((xv - mu) * rstd);
    }
    group_sum<kBwdThreads>(sum, slots);
    const float c1 = a.centre ? sum[0] * inv_n : 0.f, c2 = sum[1] * inv_n;
    for (int64_t c = threadIdx.x; c < a.n; c += kBwdThreads) {
      const float xv = load_param(x, sizeof(XT) == 4, c), gv = load_param(g, sizeof(XT) == 4, c);
      const float h = gv * (a.w ? load_param(a.w, a.w_f32, c) : 1.f);
      const float f = (h - c1 - (xv - mu) * rstd * c2) * rstd;
      if constexpr (sizeof(XT) == 4) dx[c] = f;
      else dx[c] = (uint16_t)f32_to_bf16_rne(f);
    }
    __syncthreads();
  }
}

// Wide rows, first launch: partial column sums, a workgroup per panel of 256
// columns (blockIdx.x) and slice of the rows (blockIdx.y).
template <typename XT>
__global__ __launch_bounds__(kPanel) void norm_wide_columns_kernel(NormArgs a) {
  const int64_t c = (int64_t)blockIdx.x * kPanel + threadIdx.x;
  if (c >= a.n) return;
  float dw = 0.f, db = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float xv = load_param(static_cast<const XT*>(a.x) + row * a.ldx, sizeof(XT) == 4, c), gv = load_param(static_cast<const XT*>(a.dy) + row * a.lddy, sizeof(XT) == 4, c);
    const float mu = a.centre ? a.mean[row] : 0.f;
    dw += gv * ((xv - mu) * a.rstd[row]);
    db += gv;
  }
  a.part[(int64_t)blockIdx.y * a.n + c] = dw;
  if (a.db) a.part[((int64_t)gridDim.y + blockIdx.y) * a.n + c] = db;
}

// dw (blockIdx.y = 0) and db (1): the G partial rows added, 64 columns per
// workgroup, sixteen waves each taking every sixteenth row, then in wave order.
__global__ __launch_bounds__(1024) void norm_params_kernel(const float* part, int64_t G, int64_t n, int f32, void* dw,
                                                           void* db) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  const float* p = part + (int64_t)blockIdx.y * G * n + c;
  float s = 0.f;
  if (c < n) {
#pragma unroll 8
    for (int64_t g = wave; g < G; g += 16) s += p[g * n];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < n) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sums[i][lane];
    void* out = blockIdx.y ? db : dw;
    if (f32)
      static_cast<float*>(out)[c] = s;
    else
      static_cast<uint16_t*>(out)[c] = (uint16_t)f32_to_bf16_rne(s);
  }
}

size_t elem(rgc_dtype_t t) { return t == RGC_F32 ? 4 : 2; }
bool dtype_ok(rgc_dtype_t t) { return t == RGC_BF16 || t == RGC_F32; }

rgc_status_t check_rows(const void* p, int64_t ld, int64_t n, rgc_dtype_t t) {
  if (!p) return RGC_ERR_NULL;
  if (ld < n) return RGC_ERR_SHAPE;
  if (ld > int64_t(1) << 31) return RGC_ERR_UNSUPPORTED;
  if (!aligned_to(p, elem(t))) return RGC_ERR_ALIGN;
  return RGC_OK;
}

rgc_status_t check_shape(rgc_norm_kind_t kind, rgc_dtype_t xt, rgc_dtype_t wt, int64_t rows, int64_t n) {
  if (kind != RGC_NORM_LAYER && kind != RGC_NORM_RMS) return RGC_ERR_UNSUPPORTED;
  if (!dtype_ok(xt) || !dtype_ok(wt)) return RGC_ERR_UNSUPPORTED;
  if (rows < 0 || n <= 0) return RGC_ERR_SHAPE;
  if (rows > kNormMaxRows || n > kNormMaxWidth) return RGC_ERR_UNSUPPORTED;
  return RGC_OK;
}

rgc_status_t launched() { return hipGetLastError() == hipSuccess ? RGC_OK : RGC_ERR_HIP; }

template <typename XT, int NV, int TPR, int THREADS>
void forward_launch(const NormArgs& a, hipStream_t s) {
  // bf16 rows of up to 256 threads: a workgroup to each group of rows (32768 x
  // 4096: 104 us; walking four groups each 112). Others: four rounds of
  // workgroups that walk (fp32 16384 x 4096: 107 us; a workgroup to a group 111;
  // bf16 8192 x 16384: 110 and 127). Launches stay below 2^31 threads.
  const int64_t groups = (a.rows + THREADS / TPR - 1) / (THREADS / TPR);
  const int64_t most = sizeof(XT) == 2 && THREADS == 256 ? int64_t(1) << 20 : (int64_t)device_compute_units() * (2048 / THREADS) * 4;
  const dim3 grid((unsigned)(groups < most ? groups : most));
  if (a.n % 8) hipLaunchKernelGGL((norm_forward_kernel<XT, true, NV, TPR, THREADS>), grid, dim3(THREADS), 0, s, a);
  else hipLaunchKernelGGL((norm_forward_kernel<XT, false, NV, TPR, THREADS>), grid, dim3(THREADS), 0, s, a);
}

template <typename XT>
void forward_pick(const NormArgs& a, hipStream_t s) {
  if (a.n <= 128) forward_launch<XT, 1, 16, 256>(a, s);
  else if (a.n <= 512) forward_launch<XT, 1, 64, 256>(a, s);
  else if (a.n <= 1024) forward_launch<XT, 2, 64, 256>(a, s);
  else if (a.n <= 2048) forward_launch<XT, 4, 64, 256>(a, s);
  else if (a.n <= 4096) {  // bf16 4096 x 4096: 14.8 us on 256 threads a row, 16.1 on 128; fp32 16384 x 4096: 107 and 103
    if constexpr (sizeof(XT) == 2) forward_launch<XT, 2, 256, 256>(a, s);
    else forward_launch<XT, 4, 128, 256>(a, s);
  }
  else if (a.n <= 8192) forward_launch<XT, 4, 256, 256>(a, s);
  else if (a.n <= 16384) forward_launch<XT, 2, 1024, 1024>(a, s);
  else forward_launch<XT, 8, 1024, 1024>(a, s);
}

// Rows a workgroup of the backward holds at a time (as backward_pick).
int backward_rows(int64_t n, rgc_dtype_t xt) {
  const bool f32 = xt == RGC_F32;
  if (n <= 1024) return n <= 128 ? 64 : 16;
  return (n <= 2048 ? 16 : n <= 4096 ? 8 : n <= 8192 ? 4 : 2) / (f32 ? 2 : 1);
}

// Workgroups of the backward, and so partial rows: one per compute unit, or
// fewer where the rows do not fill them.
int64_t backward_groups(int64_t rows, int64_t n, rgc_dtype_t xt) {
  const int64_t cus = device_compute_units();
  if (n > kNormHeldBackward) return rows < 64 ? rows : 64;
  const int64_t per = backward_rows(n, xt);
  const int64_t need = (rows + per - 1) / per;
  return need < cus ? need : cus;
}

template <typename XT, int NV, int TPR, int THREADS>
void backward_launch(const NormArgs& a, int64_t G, hipStream_t s) {
  const dim3 grid((unsigned)G);
  if (a.n % 8) hipLaunchKernelGGL((norm_backward_kernel<XT, true, NV, TPR, THREADS>), grid, dim3(THREADS), 0, s, a);
  else hipLaunchKernelGGL((norm_backward_kernel<XT, false, NV, TPR, THREADS>), grid, dim3(THREADS), 0, s, a);
}

template <typename XT>
void backward_pick(const NormArgs& a, int64_t G, hipStream_t s) {
  if (a.n > kNormHeldBackward) {
    // (the columns first: dX may take the place of X or dY)
    hipLaunchKernelGGL(norm_wide_columns_kernel<XT>, dim3((unsigned)((a.n + kPanel - 1) / kPanel), (unsigned)G),
                       dim3(kPanel), 0, s, a);
    const int64_t most = (int64_t)device_compute_units() * 4;
    hipLaunchKernelGGL(norm_wide_dx_kernel<XT>, dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(kBwdThreads), 0, s,
                       a);
    return;
  }
  if (a.n <= 128) return backward_launch<XT, 1, 16, 1024>(a, G, s);
  if (a.n <= 512) return backward_launch<XT, 1, 64, 1024>(a, G, s);
  if (a.n <= 1024) return backward_launch<XT, 2, 64, 1024>(a, G, s);
  if constexpr (sizeof(XT) == 2) {  // up to 64 elements to a lane
    if (a.n <= 2048) return backward_launch<XT, 4, 64, 1024>(a, G, s);
    if (a.n <= 4096) return backward_launch<XT, 8, 64, 512>(a, G, s);
    if (a.n <= 8192) return backward_launch<XT, 8, 128, 512>(a, G, s);
    backward_launch<XT, 8, 256, 512>(a, G, s);
  } else {  // up to 32
    if (a.n <= 2048) return backward_launch<XT, 4, 64, 512>(a, G, s);
    if (a.n <= 4096) return backward_launch<XT, 4, 128, 512>(a, G, s);
    if (a.n <= 8192) return backward_launch<XT, 4, 256, 512>(a, G, s);
    backward_launch<XT, 4, 512, 512>(a, G, s);
  }
}

}  // namespace
}  // namespace rgc

using namespace rgc;

extern "C" rgc_status_t rgc_layer_norm_forward(rgc_norm_kind_t kind, rgc_dtype_t xt, rgc_dtype_t wt, const void* X,
                                               int64_t ldx, const void* weight, const void* bias, double eps, void* Y,
                                               int64_t ldy, float* mean, float* rstd, int64_t rows, int64_t n,
                                               void* stream) {
  rgc_status_t st = check_shape(kind, xt, wt, rows, n);
  if (st != RGC_OK) return st;
  if (!(eps >= 0) || !((float)eps <= 3e38f)) return RGC_ERR_VALUE;
  if (rows == 0) return RGC_OK;
  if ((st = check_rows(X, ldx, n, xt)) != RGC_OK) return st;
  if ((st = check_rows(Y, ldy, n, xt)) != RGC_OK) return st;
  if (!aligned_to(weight, elem(wt)) || !aligned_to(bias, elem(wt)) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return RGC_ERR_ALIGN;
  NormArgs a{};
  a.x = X, a.w = weight, a.b = bias, a.out = Y, a.mean = mean, a.rstd = rstd;
  a.ldx = ldx, a.ldo = ldy, a.rows = rows, a.n = n, a.eps = (float)eps;
  a.w_f32 = wt == RGC_F32, a.centre = kind == RGC_NORM_LAYER;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (xt == RGC_F32) forward_pick<float>(a, s);
  else forward_pick<uint16_t>(a, s);
  return launched();
}

// The partial rows of whichever type X will have.
extern "C" size_t rgc_layer_norm_backward_workspace_size(int64_t rows, int64_t n) {
  if (rows <= 0 || n <= 0 || rows > kNormMaxRows || n > kNormMaxWidth) return 0;
  const int64_t a = backward_groups(rows, n, RGC_BF16), b = backward_groups(rows, n, RGC_F32);
  return (size_t)(a > b ? a : b) * 2 * (size_t)n * 4;
}

extern "C" rgc_status_t rgc_layer_norm_backward(rgc_norm_kind_t kind, rgc_dtype_t xt, rgc_dtype_t wt, const void* dY,
                                                int64_t lddy, const void* X, int64_t ldx, const void* weight,
                                                const float* mean, const float* rstd, void* dX, int64_t lddx,
                                                void* dweight, void* dbias, int64_t rows, int64_t n, void* ws,
                                                size_t ws_bytes, void* stream) {
  rgc_status_t st = check_shape(kind, xt, wt, rows, n);
  if (st != RGC_OK) return st;
  if (!dweight) return RGC_ERR_NULL;
  if (!aligned_to(dweight, elem(wt)) || !aligned_to(dbias, elem(wt))) return RGC_ERR_ALIGN;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 params((unsigned)((n + 63) / 64), dbias ? 2 : 1);
  if (rows == 0) {  // sums over no rows
    hipLaunchKernelGGL(norm_params_kernel, params, dim3(1024), 0, s, nullptr, (int64_t)0, n, (int)(wt == RGC_F32),
                       dweight, dbias);
    return launched();
  }
  if ((st = check_rows(dY, lddy, n, xt)) != RGC_OK) return st;
  if ((st = check_rows(X, ldx, n, xt)) != RGC_OK) return st;
  if ((st = check_rows(dX, lddx, n, xt)) != RGC_OK) return st;
  if (!rstd || (kind == RGC_NORM_LAYER && !mean)) return RGC_ERR_NULL;
  if (!aligned_to(weight, elem(wt)) || !aligned_to(mean, 4) || !aligned_to(rstd, 4)) return RGC_ERR_ALIGN;
  if (!ws || ws_bytes < rgc_layer_norm_backward_workspace_size(rows, n)) return RGC_ERR_WORKSPACE;
  if (!aligned_to(ws, 256)) return RGC_ERR_ALIGN;
  NormArgs a{};
  a.x = X, a.dy = dY, a.w = weight, a.out = dX, a.part = static_cast<float*>(ws);
  a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
  a.ldx = ldx, a.lddy = lddy, a.ldo = lddx, a.rows = rows, a.n = n;
  a.w_f32 = wt == RGC_F32, a.centre = kind == RGC_NORM_LAYER, a.db = dbias != nullptr;
  const int64_t G = backward_groups(rows, n, xt);
  if (xt == RGC_F32) backward_pick<float>(a, G, s);
  else backward_pick<uint16_t>(a, G, s);
  if ((st = launched()) != RGC_OK) return st;
  hipLaunchKernelGGL(norm_params_kernel, params, dim3(1024), 0, s, a.part, G, n, a.w_f32, dweight, dbias);
  return launched();
}
