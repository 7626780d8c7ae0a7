// The global norm of many gradients, the factor that clips them, and the
// multiplication in place.
//
//   norm = |s| sqrt(sum over all tensors of g^2),  scale = s min(1, max_norm / norm)
//
// s: a factor that the gradients are to be multiplied by anyway (1 if none). A
// norm that is not finite gives a scale of NaN, on which an AdamW step leaves its
// tensors as they are and so does the multiplication here.
//
// The squares are added in fp64: those of fp32 numbers neither overflow nor
// vanish there, and a sum of 2^34 of them is off by less than fp32's last bit.
// fp64 multiply-adds run at half the rate of fp32 ones, far above what memory
// delivers: one pass over the gradients, bound by reading them. A workgroup takes a
// chunk of one tensor and leaves one partial sum in the workspace; a last launch of one
// workgroup adds the partial sums in a fixed order, so a norm repeats bit for bit.
//
// The multiplication reads and writes the gradients once more, from the last
// chunk to the first: what the norm read last is still in the last-level cache.
// A scale of 1 writes nothing.
#include "rgc_internal.hpp"

namespace rgc {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipVector = 8;                                // elements of a load
constexpr int kClipTensors = 160;                             // of a launch: their table travels in its arguments (3.4 KB)
constexpr int64_t kClipChunk = 4 * kClipThreads * kClipVector;  // smallest chunk
constexpr int64_t kClipChunks = 8192;                         // as many chunks as keep the join short
constexpr int64_t kClipMaxElements = int64_t(1) << 34;

struct ClipArgs {
  int count;
  int64_t chunk;
  double* part;        // norm: the launch's first partial sum
  const float* scale;  // multiplication
  void* g[kClipTensors];
  int64_t n[kClipTensors];
  uint32_t base[kClipTensors + 1];  // first workgroup of each tensor
  uint8_t f32[kClipTensors];
};
static_assert(sizeof(ClipArgs) < 4096, "kernel arguments");

// The tensor of workgroup b: as many of the following tensors' first workgroups as lie at or below b.
__device__ __forceinline__ int tensor_of(const ClipArgs& a, uint32_t b) {
  const int lane = threadIdx.x & 63;
  int at = 0;
#pragma unroll
  for (int q = 0; q < (kClipTensors + 63) / 64; ++q) {
    const int i = 64 * q + lane + 1;
    at += __builtin_popcountll(__ballot(i < a.count && a.base[i < a.count ? i : 0] <= b));
  }
  return __builtin_amdgcn_readfirstlane(at);
}

// Eight elements at p, at any address.
struct Bf16x8 {
  typedef u32x4v_t any_t __attribute__((aligned(2)));
  u32x4v_t v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const any_t*>(p); }
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16); }
  __device__ __forceinline__ void store(uint16_t* p, float k) const {
    u32x4v_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32x2_to_bf16x2_rne(get(2 * i) * k, get(2 * i + 1) * k);
    *reinterpret_cast<any_t*>(p) = w;
  }
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_bits_to_f32(*p); }
  static __device__ __forceinline__ void put(uint16_t* p, float f) { *p = (uint16_t)f32_to_bf16_rne(f); }
};
struct F32x8 {
  typedef f32x4_t any_t __attribute__((aligned(4)));
  f32x4_t a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const any_t*>(p)[0];
    b = reinterpret_cast<const any_t*>(p)[1];
  }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i & 3] : b[i & 3]; }
  __device__ __forceinline__ void store(float* p, float k) const {
    reinterpret_cast<any_t*>(p)[0] = f32x4_t{a[0] * k, a[1] * k, a[2] * k, a[3] * k};
    reinterpret_cast<any_t*>(p)[1] = f32x4_t{b[0] * k, b[1] * k, b[2] * k, b[3] * k};
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float f) { *p = f; }
};

// Sum of squares of this thread's elements among `count` at p: four vectors
// at a time, then one by one what is no whole round of the workgroup.
template <typename Vec, typename T>
__device__ __forceinline__ double squares(const T* p, int64_t count) {
  constexpr int kRound = kClipThreads * kClipVector;
  double sum[4] = {0, 0, 0, 0};
  int64_t at = kClipVector * threadIdx.x;
  for (; at + 3 * kRound + kClipVector <= count; at += 4 * kRound) {
    Vec v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u].load(p + at + u * kRound);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double d = v[u].get(i);
        sum[u] = __builtin_fma(d, d, sum[u]);
      }
  }
  for (; at < count; at += kRound) {
    const int left = (int)(count - at < kClipVector ? count - at : kClipVector);
    if (left == kClipVector) {
      Vec v;
      v.load(p + at);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double d = v.get(i);
        sum[i & 3] = __builtin_fma(d, d, sum[i & 3]);
      }
    } else {
      for (int i = 0; i < left; ++i) {
        const double d = Vec::one(p + at + i);
        sum[0] = __builtin_fma(d, d, sum[0]);
      }
    }
  }
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

__global__ __launch_bounds__(kClipThreads) void clip_squares_kernel(ClipArgs a) {
  __shared__ double waves[kClipThreads / 64];
  const int i = tensor_of(a, blockIdx.x);
  const int64_t at = (int64_t)(blockIdx.x - a.base[i]) * a.chunk;
  const int64_t count = a.n[i] - at < a.chunk ? a.n[i] - at : a.chunk;
  double s = a.f32[i] ? squares<F32x8>(static_cast<const float*>(a.g[i]) + at, count)
                      : squares<Bf16x8>(static_cast<const uint16_t*>(a.g[i]) + at, count);
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) a.part[blockIdx.x] = (waves[0] + waves[1]) + (waves[2] + waves[3]);
}

// The partial sums added, and the norm and the scale.
__global__ __launch_bounds__(1024) void clip_join_kernel(const double* part, int64_t count, double max_norm,
                                                         const float* grad_scale, float* norm_out, float* scale_out) {
  __shared__ double waves[16];
  double s = 0;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < count; i += 1024) s += part[i];
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x > 0) return;
  s = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += waves[i];
  const double factor = grad_scale ? (double)*grad_scale : 1.0;
  const double norm = __builtin_fabs(factor) * sqrt(s);
  *norm_out = (float)norm;
  // (the difference is 0 for every finite number)
  *scale_out = norm - norm == 0 ? (float)(norm > max_norm ? factor * (max_norm / norm) : factor) : __builtin_nanf("");
}

template <typename Vec, typename T>
__device__ __forceinline__ void multiply(T* p, int64_t count, float k) {
  constexpr int kRound = kClipThreads * kClipVector;
  int64_t at = kClipVector * threadIdx.x;
  for (; at + 3 * kRound + kClipVector <= count; at += 4 * kRound) {
    Vec v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u].load(p + at + u * kRound);
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u].store(p + at + u * kRound, k);
  }
  for (; at < count; at += kRound) {
    const int left = (int)(count - at < kClipVector ? count - at : kClipVector);
    if (left == kClipVector) {
      Vec v;
      v.load(p + at);
      v.store(p + at, k);
    } else {
      for (int i = 0; i < left; ++i) Vec::put(p + at + i, Vec::one(p + at + i) * k);
    }
  }
}

__global__ __launch_bounds__(kClipThreads) void clip_scale_kernel(ClipArgs a) {
  const float k = *a.scale;
  if (k == 1.f || !(k - k == 0.f)) return;
  const uint32_t b = gridDim.x - 1 - blockIdx.x;
  const int i = tensor_of(a, b);
  const int64_t at = (int64_t)(b - a.base[i]) * a.chunk;
  const int64_t count = a.n[i] - at < a.chunk ? a.n[i] - at : a.chunk;
  if (a.f32[i]) multiply<F32x8>(static_cast<float*>(a.g[i]) + at, count, k);
  else multiply<Bf16x8>(static_cast<uint16_t*>(a.g[i]) + at, count, k);
}

// Elements of a workgroup: a power of two times the smallest chunk, the same for all
// tensors of a call. 0 if there are too many elements.
int64_t chunk_of(int64_t n, const int64_t* numels) {
  int64_t all = 0;
  for (int64_t i = 0; i < n; ++i) all += numels[i];
  int64_t chunk = kClipChunk;
  while (all / chunk > kClipChunks) chunk *= 2;
  return chunk;
}

int64_t chunks_of(int64_t n, const int64_t* numels, int64_t chunk) {
  int64_t count = 0;
  for (int64_t i = 0; i < n; ++i) count += (numels[i] + chunk - 1) / chunk;
  return count;
}

rgc_status_t check_tensors(int64_t n, const rgc_dtype_t* gts, const void* const* Gs, const int64_t* numels) {
  if (n < 0) return RGC_ERR_SHAPE;
  if (n > int64_t(1) << 24) return RGC_ERR_UNSUPPORTED;
  if (n > 0 && (!gts || !Gs || !numels)) return RGC_ERR_NULL;
  for (int64_t i = 0; i < n; ++i) {
    if (gts[i] != RGC_BF16 && gts[i] != RGC_F32) return RGC_ERR_UNSUPPORTED;
    if (numels[i] < 0) return RGC_ERR_SHAPE;
    if (numels[i] > kClipMaxElements) return RGC_ERR_UNSUPPORTED;
    if (numels[i] == 0) continue;
    if (!Gs[i]) return RGC_ERR_NULL;
    if (!aligned_to(Gs[i], gts[i] == RGC_F32 ? 4 : 2)) return RGC_ERR_ALIGN;
  }
  return RGC_OK;
}

// Calls launch(args, workgroups) for the tensors [from, to) in turn, as many as a launch's table
// holds; tensors without elements are left out. BACK: from the last launch to the first.
template <bool BACK, typename F>
rgc_status_t for_each_launch(int64_t n, const rgc_dtype_t* gts, const void* const* Gs, const int64_t* numels,
                             int64_t chunk, F&& launch) {
  const int64_t tables = (n + kClipTensors - 1) / kClipTensors;
  for (int64_t t = 0; t < tables; ++t) {
    const int64_t from = (BACK ? tables - 1 - t : t) * kClipTensors, to = from + kClipTensors < n ? from + kClipTensors : n;
    ClipArgs a{};
    a.chunk = chunk;
    for (int64_t i = from; i < to; ++i) {
      if (numels[i] == 0) continue;
      const int c = a.count++;
      a.g[c] = const_cast<void*>(Gs[i]), a.n[c] = numels[i], a.f32[c] = gts[i] == RGC_F32;
      a.base[c + 1] = a.base[c] + (uint32_t)((numels[i] + chunk - 1) / chunk);
    }
    if (a.count == 0) continue;
    launch(a, a.base[a.count]);
    if (hipGetLastError() != hipSuccess) return RGC_ERR_HIP;
  }
  return RGC_OK;
}

}  // namespace
}  // namespace rgc

using namespace rgc;

extern "C" size_t rgc_grad_norm_batch_workspace_size(int64_t n, const int64_t* numels) {
  if (n <= 0 || n > int64_t(1) << 24 || !numels) return 0;
  for (int64_t i = 0; i < n; ++i)
    if (numels[i] < 0 || numels[i] > kClipMaxElements) return 0;
  return (size_t)chunks_of(n, numels, chunk_of(n, numels)) * sizeof(double);
}

extern "C" rgc_status_t rgc_grad_norm_batch(int64_t n, const rgc_dtype_t* gts, const void* const* Gs,
                                            const int64_t* numels, double max_norm, const float* grad_scale, float* norm,
                                            float* scale, void* ws, size_t ws_bytes, void* stream) {
  rgc_status_t st = check_tensors(n, gts, Gs, numels);
  if (st != RGC_OK) return st;
  if (!(max_norm >= 0)) return RGC_ERR_VALUE;
  if (!norm || !scale) return RGC_ERR_NULL;
  if (!aligned_to(norm, 4) || !aligned_to(scale, 4) || !aligned_to(grad_scale, 4)) return RGC_ERR_ALIGN;
  const int64_t chunk = chunk_of(n, numels), chunks = chunks_of(n, numels, chunk);
  if (chunks > 0 && (!ws || ws_bytes < (size_t)chunks * sizeof(double))) return RGC_ERR_WORKSPACE;
  if (!aligned_to(ws, 256)) return RGC_ERR_ALIGN;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  double* part = static_cast<double*>(ws);
  st = for_each_launch<false>(n, gts, Gs, numels, chunk, [&](ClipArgs& a, uint32_t blocks) {
    a.part = part;
    part += blocks;
    hipLaunchKernelGGL(clip_squares_kernel, dim3(blocks), dim3(kClipThreads), 0, s, a);
  });
  if (st != RGC_OK) return st;
  hipLaunchKernelGGL(clip_join_kernel, dim3(1), dim3(1024), 0, s, static_cast<const double*>(ws), chunks, max_norm,
                     grad_scale, norm, scale);
  return hipGetLastError() == hipSuccess ? RGC_OK : RGC_ERR_HIP;
}

extern "C" rgc_status_t rgc_scale_batch(int64_t n, const rgc_dtype_t* gts, void* const* Gs, const int64_t* numels,
                                        const float* scale, void* stream) {
  const rgc_status_t st = check_tensors(n, gts, Gs, numels);
  if (st != RGC_OK || n == 0) return st;
  if (!scale) return RGC_ERR_NULL;
  if (!aligned_to(scale, 4)) return RGC_ERR_ALIGN;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return for_each_launch<true>(n, gts, Gs, numels, chunk_of(n, numels), [&](ClipArgs& a, uint32_t blocks) {
    a.scale = scale;
    hipLaunchKernelGGL(clip_scale_kernel, dim3(blocks), dim3(kClipThreads), 0, s, a);
  });
}
