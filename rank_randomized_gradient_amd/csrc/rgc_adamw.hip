// One AdamW step over many tensors, with moments in fp32 or in 8 bits:
//
//   g' = scale g,  m <- b1 m + (1 - b1) g',  v <- b2 v + (1 - b2) g'^2
//   p <- p - (lr wd p + lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps))
//
// in fp32 whatever the stored types. Both terms are joined before the one
// subtraction: a factor 1 - lr wd rounded to fp32 would be 1 at lr wd = 1e-8 and
// decay twice as fast as asked at 3e-8. bf16 parameters are rounded
// stochastically, as the sketched update's weights are: no fp32 copy is kept,
// and a step far below half a unit in the last place still moves the weight
// in expectation.
//
// 8-bit moments: m and sqrt(v) are e4m3 values in blocks of 128 with one
// power-of-two scale each, chosen so that the block's largest finite magnitude
// lies in 128 .. 256 units (below e4m3's largest, 448). Powers of two make the
// scaling exact, so the only error is the rounding to four significant bits.
// A moment that moves by less than half a step of its code stands still if it is
// rounded to nearest, whatever moves it. sqrt(v) changes by at most (1 - b2) / 2
// of itself while the gradient is small, and so would never decay: it is rounded
// stochastically. m changes by up to 1 - b1 of itself, and half a step is 1/30 to
// 1/16 of it: at b1 = 0.9 a block of zero gradients still decays to nothing, at
// 0.95 it does not, and m / sqrt(v) of a parameter that should stand still grows
// without end; under a constant gradient m stops short of it, at 0.72 of it for b1 =
// 0.9, 0.54 for 0.95, 0.19 for 0.99 (means over random gradients). So m is rounded
// stochastically too (STOCHASTIC), which keeps its mean. Rounding it to nearest is
// the other form, up to b1 = 0.9; there an element whose gradients end beside live
// ones keeps four subnormal steps of its block, 2^-14 of the block's largest.
// A sqrt(v) that is not zero never rounds to zero, since a zero one under a
// momentum that is not zero would leave eps alone to divide by. Infinities and NaN
// become NaN codes and are left out of the scale: they spoil their own elements only.
//
// Bound by memory: 2 p + g + 16 bytes an element in fp32 states, 2 p + g + 4
// in 8 bits (10 bytes for bf16). 134M bf16 parameters with 8-bit states take 248
// us on MI355X (5.4 TB/s; a copy reaches 5.2; 238 on the same tensors step after
// step, with m rounded either way), 60 ragged fp32 ones of 29M elements with fp32
// states 161 us (5.1 TB/s). With a correctly rounded division and square root and every
// element checked for NaN the 8-bit step took 283 us, bound by instructions.
// Eight consecutive elements to a thread, so
// one Philox call (128 bits) serves the thread: element j of the eight takes
// half j % 2 of word j / 2 for its parameter, the other half, its neighbour's, for
// its second moment and half j % 2 of the next word (the first after the last) for
// its first, which makes an element's rounding errors independent of each other. A block of 128 is sixteen lanes, so its
// maxima are lane rotations within a row of sixteen.
#include <math.h>

#include "rgc_internal.hpp"

namespace rgc {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamChunk = kAdamThreads * 8;  // elements of a workgroup
constexpr int kAdamTensors = 48;              // tensors of a launch: their table travels in the kernel's arguments
constexpr uint32_t kTagAdam = 4;              // counter word 2 of the rounding bits

struct AdamTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t n;
};

struct AdamArgs {
  int count;
  uint32_t first;  // index of the launch's first tensor within the call
  uint32_t key0, key1;
  float b1, c1, b2, c2;  // b1, 1 - b1, b2, 1 - b2
  float decay;           // lr wd
  float size;            // lr / (1 - b1^t)
  float root;            // 1 / sqrt(1 - b2^t)
  float eps;
  const float* scale;  // gradients' factor, or null
  uint32_t base[kAdamTensors + 1];  // first workgroup of each tensor
  AdamTensor t[kAdamTensors];
};

__device__ __forceinline__ void load8(const float* p, int64_t at, int count, float (&f)[8]) {
  if (count == 8) {
    const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p + at), b = *reinterpret_cast<const f32x4_t*>(p + at + 4);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j < count ? p[at + j] : 0.f;
  }
}
__device__ __forceinline__ void load8(const uint16_t* p, int64_t at, int count, float (&f)[8]) {
  if (count == 8) {
    const u32x4v_t a = *reinterpret_cast<const u32x4v_t*>(p + at);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j < count ? bf16_bits_to_f32(p[at + j]) : 0.f;
  }
}
__device__ __forceinline__ void store8(float* p, int64_t at, int count, const float (&f)[8]) {
  if (count == 8) {
    *reinterpret_cast<f32x4_t*>(p + at) = f32x4_t{f[0], f[1], f[2], f[3]};
    *reinterpret_cast<f32x4_t*>(p + at + 4) = f32x4_t{f[4], f[5], f[6], f[7]};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < count) p[at + j] = f[j];
  }
}

// Eight e4m3 codes (two dwords) and their values.
__device__ __forceinline__ void load_codes(const uint8_t* p, int64_t at, int count, float unit, float (&f)[8]) {
  uint32_t w[2] = {0u, 0u};
  if (count == 8) {
    const u32x2v_t a = *reinterpret_cast<const u32x2v_t*>(p + at);
    w[0] = a.x, w[1] = a.y;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < count) w[j / 4] |= (uint32_t)p[at + j] << (8 * (j & 3));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
    f[4 * h] = lo[0] * unit, f[4 * h + 1] = lo[1] * unit, f[4 * h + 2] = hi[0] * unit, f[4 * h + 3] = hi[1] * unit;
  }
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t at, int count, const float (&f)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int q = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h], f[4 * h + 1], 0, false);
    w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2], f[4 * h + 3], q, true);
  }
  if (count == 8) {
    *reinterpret_cast<u32x2v_t*>(p + at) = u32x2v_t{w[0], w[1]};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < count) p[at + j] = (uint8_t)(w[j / 4] >> (8 * (j & 3)));
  }
}

// Maximum over the sixteen lanes of a row, in all of them: rotations by 8, 4, 2, 1.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  const auto turned = [](uint32_t x, auto r) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + decltype(r)::value, 0xF, 0xF, false);
  };
  const auto up = [&](uint32_t x, auto r) {
    const uint32_t y = turned(x, r);
    return x > y ? x : y;
  };
  return up(up(up(up(v, IntC<8>{}), IntC<4>{}), IntC<2>{}), IntC<1>{});
}

constexpr uint32_t kInfBits = 0x7F800000u;
__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & kInfBits) != kInfBits; }

// Largest of eight magnitudes as bits, which order magnitudes as they are and
// NaN above infinity: one comparison of the result tells whether all are finite.
__device__ __forceinline__ uint32_t top_bits(const float (&f)[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = __float_as_uint(f[j]) & 0x7FFFFFFFu;
    m = m > b ? m : b;
  }
  return m;
}

// sqrt(v) for v from 2^-100 up to infinity, not included: v rsq(v), and one
// step s + (v - s^2) / (2 s) with the residual exact in an fma, which leaves
// the correctly rounded root but for values within 2^-20 of a half step.
__device__ __forceinline__ float plain_root(float v) {
  const float r = __builtin_amdgcn_rsqf(v), s = v * r;
  return __builtin_fmaf(__builtin_fmaf(-s, s, v), 0.5f * r, s);
}

// Exponent field of the unit that brings `top` into 128 .. 256, at least 1
// (2^-126, the smallest normal number, for a block of zeros too).
__device__ __forceinline__ uint32_t unit_exponent(uint32_t top) {
  const int e = (int)(top >> 23) - 7;
  return (uint32_t)(e < 1 ? 1 : e);
}

// Eight numbers of magnitude below 256 rounded to e4m3 values with the 16 random
// bits r[j] each: three bits of mantissa, the 20 below them rounded by the random
// ones (a carry goes up through the magnitude; the sign bit is out of reach).
// e4m3's subnormals have the step of its smallest normal numbers, 2^-9, so what
// lies below 2^-6 is rounded lifted by that much, where fp32 truncates at that
// step. Whether a lane of the wave held such a number.
__device__ __forceinline__ bool round_codes(float (&q)[8], const uint32_t (&r)[8]) {
  bool small = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) small |= !(fabsf(q[j]) >= 0.015625f);
  if (__any(small)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = fabsf(q[j]), lift = x < 0.015625f ? 0.015625f : 0.f;
      const float y = __uint_as_float((__float_as_uint(x + lift) + (r[j] << 4)) & 0xFFF00000u) - lift;
      q[j] = copysignf(y, q[j]);
    }
    return true;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = __uint_as_float((__float_as_uint(q[j]) + (r[j] << 4)) & 0xFFF00000u);
  return false;
}

template <typename PT, typename GT, bool EIGHT, bool STOCHASTIC>
__global__ __launch_bounds__(kAdamThreads) void adamw_kernel(AdamArgs a) {
  const float scale = a.scale ? *a.scale : 1.f;
  if (!finite(scale)) return;  // gradients that overflowed: the step is skipped
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {  // the last tensor whose first workgroup is not behind this one
    const int mid = (lo + hi + 1) / 2;
    if (a.base[mid] <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const AdamTensor& t = a.t[lo];
  const int64_t at = (int64_t)(blockIdx.x - a.base[lo]) * kAdamChunk + (int64_t)threadIdx.x * 8;
  const int64_t left = t.n - at;
  const int count = left >= 8 ? 8 : left > 0 ? (int)left : 0;  // 0: past the end, but still a lane of its block's maxima
  PT* P = static_cast<PT*>(t.p);
  float p[8], g[8], m[8], v[8];
  load8(P, at, count, p);
  load8(static_cast<const GT*>(t.g), at, count, g);
  const int64_t block = at / 128;
  const bool any = block * 128 < t.n;
  if constexpr (EIGHT) {
    load_codes(static_cast<const uint8_t*>(t.m), at, count, any ? t.ms[block] : 0.f, m);
    load_codes(static_cast<const uint8_t*>(t.v), at, count, any ? t.vs[block] : 0.f, v);
  } else {
    load8(static_cast<const float*>(t.m), at, count, m);
    load8(static_cast<const float*>(t.v), at, count, v);
  }
  // Infinities, NaN, zeros and subnormal numbers take the careful path, with
  // their whole wave; the other has half the instructions.
  float root[8];
  uint32_t low = ~0u, high = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    g[j] = g[j] * scale;
    m[j] = m[j] * a.b1 + g[j] * a.c1;
    if constexpr (EIGHT) v[j] = v[j] * v[j];
    v[j] = v[j] * a.b2 + g[j] * g[j] * a.c2;
    const uint32_t b = __float_as_uint(v[j]);
    low = low < b ? low : b;
    high = high > b ? high : b;
  }
  if (__any(low < (27u << 23) || high >= kInfBits)) {  // 2^-100
#pragma unroll
    for (int j = 0; j < 8; ++j) root[j] = sqrtf(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) root[j] = plain_root(v[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {  // (the reciprocal is good to one unit in the last place)
    // an infinite parameter's decay is finite, or infinity would be subtracted from itself
    const float d = __builtin_amdgcn_fmed3f(p[j], -0x1.fffffep127f, 0x1.fffffep127f) * a.decay;
    p[j] = p[j] - (d + a.size * (m[j] * __builtin_amdgcn_rcpf(root[j] * a.root + a.eps)));
  }
  u32x4 bits{0u, 0u, 0u, 0u};
  if constexpr (EIGHT || sizeof(PT) == 2) {
    const uint64_t group = (uint64_t)at / 8;
    bits = philox4x32_10(u32x4{(uint32_t)group, (uint32_t)(group >> 32), kTagAdam, a.first + (uint32_t)lo}, a.key0, a.key1);
  }
  const uint32_t word[4] = {bits.x, bits.y, bits.z, bits.w};
  if constexpr (sizeof(PT) == 2) {
    if (count == 8) {
      u32x4v_t w;
      if (__any(top_bits(p) > kInfBits)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = f32x2_to_bf16x2_sr(p[2 * j], p[2 * j + 1], word[j]);
      } else {  // no NaN: the sum's high half as it is
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = __builtin_amdgcn_perm(__float_as_uint(p[2 * j + 1]) + (word[j] >> 16),
                                       __float_as_uint(p[2 * j]) + (word[j] & 0xFFFFu), 0x07060302u);
      }
      *reinterpret_cast<u32x4v_t*>(P + at) = w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < count) P[at + j] = (uint16_t)f32_to_bf16_sr(p[j], j & 1 ? word[j / 2] >> 16 : word[j / 2] & 0xFFFFu);
    }
  } else {
    store8(P, at, count, p);
  }
  if constexpr (EIGHT) {
    uint32_t mt = top_bits(m), vt = top_bits(root);
    const bool wild = __any(mt >= kInfBits || vt >= kInfBits);
    if (wild) {
      mt = vt = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t mb = finite(m[j]) ? __float_as_uint(m[j]) & 0x7FFFFFFFu : 0u;
        const uint32_t vb = finite(root[j]) ? __float_as_uint(root[j]) & 0x7FFFFFFFu : 0u;
        mt = mt > mb ? mt : mb;
        vt = vt > vb ? vt : vb;
      }
    }
    const uint32_t me = unit_exponent(row_max(mt)), ve = unit_exponent(row_max(vt));
    const float im = __uint_as_float((254u - me) << 23), iv = __uint_as_float((254u - ve) << 23);  // 1 / unit
    float qm[8], qv[8];
    uint32_t rm[8], rv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      qm[j] = m[j] * im;
      qv[j] = root[j] * iv;
      const uint32_t next = word[(j / 2 + 1) & 3];
      rm[j] = j & 1 ? next >> 16 : next & 0xFFFFu;
      rv[j] = j & 1 ? word[j / 2] & 0xFFFFu : word[j / 2] >> 16;
    }
    if constexpr (STOCHASTIC) round_codes(qm, rm);
    if (round_codes(qv, rv)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) qv[j] = root[j] > 0.f ? fmaxf(qv[j], 0.001953125f) : 0.f;
    }
    if (wild) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float nan = __uint_as_float(0x7FC00000u);
        if (!finite(m[j])) qm[j] = nan;
        if (!finite(root[j])) qv[j] = nan;
      }
    }
    store_codes(static_cast<uint8_t*>(t.m), at, count, qm);
    store_codes(static_cast<uint8_t*>(t.v), at, count, qv);
    if (any && (threadIdx.x & 15) == 0) {
      t.ms[block] = __uint_as_float(me << 23);
      t.vs[block] = __uint_as_float(ve << 23);
    }
  } else {
    store8(static_cast<float*>(t.m), at, count, m);
    store8(static_cast<float*>(t.v), at, count, v);
  }
}

template <typename PT, typename GT>
void launch(const AdamArgs& a, bool eight, bool stochastic, hipStream_t s) {
  const dim3 grid(a.base[a.count]);
  if (!eight) hipLaunchKernelGGL((adamw_kernel<PT, GT, false, false>), grid, dim3(kAdamThreads), 0, s, a);
  else if (stochastic) hipLaunchKernelGGL((adamw_kernel<PT, GT, true, true>), grid, dim3(kAdamThreads), 0, s, a);
  else hipLaunchKernelGGL((adamw_kernel<PT, GT, true, false>), grid, dim3(kAdamThreads), 0, s, a);
}

bool dtype_ok(rgc_dtype_t t) { return t == RGC_BF16 || t == RGC_F32; }

}  // namespace
}  // namespace rgc

using namespace rgc;

extern "C" rgc_status_t rgc_adamw_batch_with(unsigned flags, int64_t n, rgc_dtype_t pt, rgc_dtype_t gt, int state_bits,
                                             void* const* Ps, const void* const* Gs, void* const* Ms, void* const* Vs,
                                             float* const* Mscales, float* const* Vscales, const int64_t* numels,
                                             double lr, double beta1, double beta2, double eps, double weight_decay,
                                             int64_t step, const float* grad_scale, uint64_t seed, void* stream) {
  if (n < 0) return RGC_ERR_SHAPE;
  if (!dtype_ok(pt) || !dtype_ok(gt) || (state_bits != 8 && state_bits != 32) || n > INT32_MAX ||
      (flags & ~(unsigned)(RGC_ADAMW_STOCHASTIC_M | RGC_ADAMW_CHECK_ONLY)))
    return RGC_ERR_UNSUPPORTED;
  const bool stochastic = (flags & RGC_ADAMW_STOCHASTIC_M) != 0;
  // scalars that would divide by zero or give values that are not finite for finite inputs
  if (!(fabs(lr) <= 1e30) || !(beta1 >= 0 && (float)beta1 < 1) || !(beta2 >= 0 && (float)beta2 < 1) || !(eps <= 1e30) ||
      !((float)eps >= 0x1p-126f) || !(fabs(weight_decay) <= 1e30) || !(fabs(lr * weight_decay) <= 1e30) || step < 1 ||
      !(fabs(lr) <= 1e30 * (1 - pow(beta1, (double)step))))
    return RGC_ERR_VALUE;
  // a first moment that rounding to nearest would hold in place
  if (state_bits == 8 && !stochastic && beta1 > 0.9) return RGC_ERR_VALUE;
  if (n == 0) return RGC_OK;
  const bool eight = state_bits == 8;
  if (!Ps || !Gs || !Ms || !Vs || !numels || (eight && (!Mscales || !Vscales))) return RGC_ERR_NULL;
  if (!aligned_to(grad_scale, 4)) return RGC_ERR_ALIGN;
  for (int64_t i = 0; i < n; ++i) {
    if (numels[i] < 0) return RGC_ERR_SHAPE;
    if (numels[i] > int64_t(1) << 34) return RGC_ERR_UNSUPPORTED;
    if (numels[i] == 0) continue;
    if (!Ps[i] || !Gs[i] || !Ms[i] || !Vs[i] || (eight && (!Mscales[i] || !Vscales[i]))) return RGC_ERR_NULL;
    if (!aligned16(Ps[i]) || !aligned16(Gs[i]) || !aligned16(Ms[i]) || !aligned16(Vs[i]) ||
        (eight && (!aligned_to(Mscales[i], 4) || !aligned_to(Vscales[i], 4))))
      return RGC_ERR_ALIGN;
  }
  if (flags & RGC_ADAMW_CHECK_ONLY) return RGC_OK;
  AdamArgs a{};
  a.key0 = (uint32_t)seed, a.key1 = (uint32_t)(seed >> 32);
  a.b1 = (float)beta1, a.c1 = (float)(1 - beta1), a.b2 = (float)beta2, a.c2 = (float)(1 - beta2);
  a.decay = (float)(lr * weight_decay);
  a.size = (float)(lr / (1 - pow(beta1, (double)step)));
  a.root = (float)(1 / sqrt(1 - pow(beta2, (double)step)));
  a.eps = (float)eps;
  a.scale = grad_scale;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  // launches of up to kAdamTensors consecutive tensors and 2^23 workgroups (2^31 threads)
  for (int64_t i = 0; i < n;) {
    a.first = (uint32_t)i;
    a.count = 0;
    uint64_t groups = 0;
    while (i < n && a.count < kAdamTensors) {
      const uint64_t need = ((uint64_t)numels[i] + kAdamChunk - 1) / kAdamChunk;
      if (a.count > 0 && groups + need > (uint64_t(1) << 23)) break;
      AdamTensor& t = a.t[a.count];
      t.p = Ps[i], t.g = Gs[i], t.m = Ms[i], t.v = Vs[i], t.n = numels[i];
      t.ms = eight ? Mscales[i] : nullptr, t.vs = eight ? Vscales[i] : nullptr;
      a.base[a.count++] = (uint32_t)groups;
      groups += need;
      ++i;
    }
    a.base[a.count] = (uint32_t)groups;
    if (groups == 0) continue;
    if (pt == RGC_F32) {
      if (gt == RGC_F32) launch<float, float>(a, eight, stochastic, s);
      else launch<float, uint16_t>(a, eight, stochastic, s);
    } else {
      if (gt == RGC_F32) launch<uint16_t, float>(a, eight, stochastic, s);
      else launch<uint16_t, uint16_t>(a, eight, stochastic, s);
    }
    if (hipGetLastError() != hipSuccess) return RGC_ERR_HIP;
  }
  return RGC_OK;
}

extern "C" rgc_status_t rgc_adamw_batch(int64_t n, rgc_dtype_t pt, rgc_dtype_t gt, int state_bits, void* const* Ps,
                                        const void* const* Gs, void* const* Ms, void* const* Vs, float* const* Mscales,
                                        float* const* Vscales, const int64_t* numels, double lr, double beta1,
                                        double beta2, double eps, double weight_decay, int64_t step,
                                        const float* grad_scale, uint64_t seed, void* stream) {
  return rgc_adamw_batch_with(0, n, pt, gt, state_bits, Ps, Gs, Ms, Vs, Mscales, Vscales, numels, lr, beta1, beta2, eps,
                              weight_decay, step, grad_scale, seed, stream);
}
