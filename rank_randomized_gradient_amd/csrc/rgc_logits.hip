// Log probabilities of given tokens, entropies and the most likely alternatives
// of rows of logits, and the gradient of the first two.
//
//   lse = m + log s,  s = sum exp(z - m),  m = max z
//   logp = z_y - m - log s,  H = log s - q / s,  q = sum exp(z - m) (z - m)
//   dz_v = p_v (-gl - ge (z_v - lse + H)) + gl [v = y],  p = exp(z - lse)
//
// Entries of -inf have no probability: they add nothing to s and q and get no
// gradient but the token's own gl, which it gets whatever its logit. A row of nothing
// else has lse = -inf, a log probability of -inf, an entropy of 0 and no gradient at all.
// NaN and +inf make their row NaN.
//
// Both directions are bound by memory: the forward reads a row once, the
// backward reads and writes it once. MI355X, 4096 x 131072 bf16: forward 201 us (5.3 TB/s;
// a copy reaches 5.2), with 8, 20 and 64 alternatives 218, 224 and 278, backward 385 us (5.6 TB/s).
// Sorted lists in the lanes' registers, an insertion an entry, took 260, 313 and 548 us.
//
// The backward's z - lse loses log s where lse is large (a row of the type's
// lowest value throughout: its probabilities would be 1 each). From |lse| = 1024 on, where
// half a step of lse is 2^-14, it makes m and log s anew and takes z - m - log s.
//
// Forward: a workgroup takes a row, or one of several parts of it where there are
// few rows; a second launch then joins the parts. Every thread keeps its own
// maximum and its two sums against it, brought to the new maximum once for every
// batch of vectors it reads. A term's exponent is one multiply-add, z log2 e - m log2 e, whose
// second part is rounded once for all terms and put right at the end. (So for a wave whose
// largest entry lies within 8192 of zero; one beyond, a mask of the type's lowest value say, is
// read again and takes z - m. A thread's entries below -8192 are taken against -8192.)
//
// Alternatives: an entry's key is its value's bits in an order of unsigned numbers,
// then the complement of its index, in 64 bits: no two keys are equal, and of equal values the
// lowest index comes first. A wave keeps the keys that may be among the row's `top`
// in a small list in LDS, in any order. An entry is looked at only if it reaches a
// bar that `top` entries already reach: every lane's largest so far is an entry of its own, so
// ceil(top / 4) of a wave's 64 lanes reach a number found bit by bit, and the least of the
// four waves' numbers is the bar (below 4 alternatives the largest number that `top` of a wave's lanes reach). It is
// raised after 1, 2, 4, .. batches, so that a row of n entries lists about top (1 +
// log(n / 8192)) of them; where rows tie at the bar and the list fills, it
// is cut down to its own `top`, and keys decide from then on. At the end
// each listed key's place is the number of larger ones, counted by a thread of its own.
// The slow orders (1024 x 131072 bf16 without alternatives, with 8 and with 64; random rows take 57, 61 and 88 us): where
// entries rise along the row all that follow the last raise pass the bar, and the list is cut for every 64 of
// them: 48, 541 and 1545 us; a row whose largest entry lies beyond 8192 is read twice, by a vector's elements the second
// time: 185, 208 and 229.
#include <math.h>

#include "rgc_internal.hpp"

namespace rgc {
namespace {

constexpr int64_t kLpMaxVocab = int64_t(1) << 24;
constexpr int64_t kLpMaxRows = int64_t(1) << 31;
constexpr int64_t kLpMaxLeadingDim = int64_t(1) << 31;
constexpr int kLpMaxTop = 64;
constexpr int kLpThreads = 256;
constexpr int kLpWaves = kLpThreads / 64;
constexpr int kLpBatch = 4;                              // vectors of eight that a thread reads together
constexpr int kLpRound = kLpThreads * 8 * kLpBatch;      // entries of a workgroup's batch
constexpr int64_t kLpMaxParts = 64;
constexpr int kLpList = 128;                             // keys of a wave: `top` of them and one of each lane
constexpr int kLpJoinThreads = 512;
static_assert(kLpMaxTop + 64 <= kLpList, "a list cut down takes a key of every lane");
constexpr float kLpFloor = -200.f;  // least z - m in a product with its exponential, which is 0 from -104 on
constexpr float kLpFar = 1024.f;       // of lse: see above
constexpr float kLpLog2e = 1.4426950408889634f, kLpLn2 = 0.6931471805599453f;
constexpr float kLpFloor2 = -300.f;  // kLpFloor in units of 2
constexpr float kLpNear = 8192.f;    // of a wave's largest: its product with log2 e is off by 2^-11 at most

typedef unsigned long long u64;

struct LpArgs {
  const void* z;
  int64_t ldz, rows;
  int V, top;
  int parts;           // of a row
  int part;            // entries of a part, a multiple of 8
  const int64_t* tokens;
  float* logp;
  float* entropy;
  float* lse;
  float* top_logp;
  int64_t* top_ids;
  f32x4_t* sums;       // parts > 1: (m, s, q) of each
  u64* keys;           // parts > 1: top of each
  // backward
  void* dz;
  int64_t lddz;
  const float* grad_logp;
  const float* grad_entropy;
};

__device__ __forceinline__ float lp_exp(float x) { return __builtin_amdgcn_exp2f(x * kLpLog2e); }

// Eight logits as loaded.
template <typename ZT>
struct LpVec;
template <>
struct LpVec<uint16_t> {
  typedef u32x4v_t any_t __attribute__((aligned(2)));
  u32x4v_t v;
  __device__ __forceinline__ void none() { v = u32x4v_t{0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u}; }
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const any_t*>(p); }
  __device__ __forceinline__ void load_some(const uint16_t* p, int count) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < count) v[i / 2] = i & 1 ? (v[i / 2] & 0xFFFFu) | (uint32_t)p[i] << 16 : (v[i / 2] & 0xFFFF0000u) | p[i];
  }
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16); }
  // hides that the elements are those of before, so that they are unpacked anew and not kept
  __device__ __forceinline__ void again() { asm volatile("" : "+v"(v)); }
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_bits_to_f32(*p); }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&f)[8]) {
    *reinterpret_cast<any_t*>(p) = u32x4v_t{f32x2_to_bf16x2_rne(f[0], f[1]), f32x2_to_bf16x2_rne(f[2], f[3]),
                                            f32x2_to_bf16x2_rne(f[4], f[5]), f32x2_to_bf16x2_rne(f[6], f[7])};
  }
  static __device__ __forceinline__ void put(uint16_t* p, float f) { *p = (uint16_t)f32_to_bf16_rne(f); }
};
template <>
struct LpVec<float> {
  typedef f32x4_t any_t __attribute__((aligned(4)));
  f32x4_t a, b;
  __device__ __forceinline__ void none() { a = b = f32x4_t{-INFINITY, -INFINITY, -INFINITY, -INFINITY}; }
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
  __device__ __forceinline__ void again() { asm volatile("" : "+v"(a), "+v"(b)); }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
    reinterpret_cast<any_t*>(p)[0] = f32x4_t{f[0], f[1], f[2], f[3]};
    reinterpret_cast<any_t*>(p)[1] = f32x4_t{f[4], f[5], f[6], f[7]};
  }
  static __device__ __forceinline__ void put(float* p, float f) { *p = f; }
};

// The value's bits in an order of unsigned numbers: -0 is 0, and every NaN lies above infinity.
__device__ __forceinline__ uint32_t order_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return __builtin_isnan(z) ? 0xFFFFFFFFu : o;
}
__device__ __forceinline__ float value_of(uint32_t order) {
  return __uint_as_float(order & 0x80000000u ? order ^ 0x80000000u : ~order);
}
__device__ __forceinline__ u64 key_of(float z, int index) { return (u64)order_of(z) << 32 | (uint32_t)~index; }

// How many of the keys list[0 .. count) are larger than a key.
__device__ __forceinline__ int place_of(u64 key, const u64* list, int count) {
  int place = 0;
#pragma unroll 4
  for (int i = 0; i < count; ++i) place += list[i] > key;
  return place;
}

// Cuts a wave's list down to its `top` largest keys, in descending order; the last of them if there are as many, else 0.
__device__ __forceinline__ u64 cut_list(u64* list, int& count, int top) {
  const int lane = threadIdx.x & 63;
  const u64 a = lane < count ? list[lane] : 0, b = 64 + lane < count ? list[64 + lane] : 0;
  const int pa = place_of(a, list, count), pb = place_of(b, list, count);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // every lane has read the list
  if (lane < count && pa < top) list[pa] = a;
  if (64 + lane < count && pb < top) list[pb] = b;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  count = count < top ? count : top;
  return count == top ? list[top - 1] : 0;
}

// A number in LDS that other waves read or write meanwhile: whatever its latest value.
__device__ __forceinline__ uint32_t get_shared(const uint32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ void put_shared(uint32_t* p, uint32_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}

// The largest number of sixteen bits that `want` of the lanes' numbers reach (0 if there is none).
__device__ __forceinline__ uint32_t reached(uint32_t mine, int want) {
  uint32_t t = 0;
#pragma unroll
  for (int bit = 15; bit >= 0; --bit) {
    const uint32_t next = t | 1u << bit;
    if (__builtin_popcountll(__ballot(mine >= next)) >= want) t = next;
  }
  return t;
}

// Joins (m, s, q) with another's: all sums against the larger maximum.
__device__ __forceinline__ void join_sums(float& m, float& s, float& q, float m1, float s1, float q1) {
  const float top = fmaxf(m, m1), base = top == -INFINITY ? 0.f : top;
  const float d0 = m - base, d1 = m1 - base, f0 = lp_exp(d0), f1 = lp_exp(d1);
  q = __builtin_fmaf(s, fmaxf(d0, kLpFloor), q) * f0 + __builtin_fmaf(s1, fmaxf(d1, kLpFloor), q1) * f1;
  s = s * f0 + s1 * f1;
  m = top;
}

// What a row gives beside its alternatives, from its sums; zy: its token's logit.
__device__ __forceinline__ void finish_row(const LpArgs& a, int64_t row, int64_t y, float zy, float m, float s, float q) {
  const bool empty = m == -INFINITY && s == 0.f;
  const float ls = logf(s), h = ls - q / s;
  const bool live = !a.tokens || (y >= 0 && y < a.V);
  a.lse[row] = empty ? -INFINITY : m + ls;
  if (a.tokens) a.logp[row] = live ? (empty ? -INFINITY : zy - m - ls) : 0.f;
  a.entropy[row] = !live || empty || h < 0.f ? 0.f : h;  // (rounding can take it below 0; NaN stays)
}
__device__ __forceinline__ void put_alternative(const LpArgs& a, int64_t row, int place, u64 key, float m, float s) {
  const bool empty = m == -INFINITY && s == 0.f;
  a.top_logp[row * a.top + place] = empty ? -INFINITY : value_of((uint32_t)(key >> 32)) - m - logf(s);
  a.top_ids[row * a.top + place] = (uint32_t)~(uint32_t)key;
}

template <typename ZT>
__device__ __forceinline__ float token_logit(const LpArgs& a, int64_t row, int64_t y) {
  return y >= 0 && y < a.V ? LpVec<ZT>::one(static_cast<const ZT*>(a.z) + row * a.ldz + y) : 0.f;
}

template <typename ZT, bool TOP>
__global__ __launch_bounds__(kLpThreads, TOP ? 6 : 1) void lp_forward_kernel(LpArgs a) {
  __shared__ __attribute__((aligned(16))) u64 lists[TOP ? kLpWaves : 1][kLpList];
  __shared__ int counts[kLpWaves];
  __shared__ uint32_t reach[kLpWaves];  // what ceil(top / 4) of each wave's lanes reach (below 4 alternatives, `top`)
  __shared__ f32x4_t sums[kLpWaves];
  const int lane = threadIdx.x & 63, wave = wave_index();
  const int64_t jobs = a.rows * a.parts;
  for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
    const int64_t row = job / a.parts;
    const int first = (int)(job - row * a.parts) * a.part;
    const int end = a.V - first < a.part ? a.V : first + a.part;
    const ZT* z = static_cast<const ZT*>(a.z) + row * a.ldz;
    int64_t y = -1;
    float zy = 0.f;
    if (threadIdx.x == 0 && a.parts == 1 && a.tokens) {  // (here, so that nothing waits for it at the end)
      y = a.tokens[row];
      zy = token_logit<ZT>(a, row, y);
    }
    // the largest so far, and the sums of 2^(z log2 e - base) against base = m log2 e as rounded, m near zero
    float peak = -INFINITY, m = -kLpNear, base = m * kLpLog2e, s = 0.f, q = 0.f;
    u64 limit = 0;  // a key at or below it is not among the row's `top`
    int count = 0;
    for (int c0 = first; c0 < end; c0 += kLpRound) {
      LpVec<ZT> v[kLpBatch];
      const int c = c0 + 8 * (int)threadIdx.x;
      if (c0 + kLpRound <= end) {
#pragma unroll
        for (int u = 0; u < kLpBatch; ++u) v[u].load(z + c + u * (8 * kLpThreads));
      } else {
#pragma unroll
        for (int u = 0; u < kLpBatch; ++u) {
          const int at = c + u * (8 * kLpThreads);
          v[u].none();
          if (at + 8 <= end) v[u].load(z + at);
          else if (at < end) v[u].load_some(z + at, end - at);
        }
      }
      float high[kLpBatch];
#pragma unroll
      for (int u = 0; u < kLpBatch; ++u) {
        high[u] = -INFINITY;
#pragma unroll
        for (int e = 0; e < 8; ++e) high[u] = fmaxf(high[u], v[u].get(e));
        peak = fmaxf(peak, high[u]);
      }
      {
        m = fminf(fmaxf(peak, -kLpNear), kLpNear);
        const float d0 = base - m * kLpLog2e, f0 = __builtin_amdgcn_exp2f(d0);
        q = __builtin_fmaf(s, fmaxf(d0, kLpFloor2), q) * f0;
        s *= f0;
        base = m * kLpLog2e;
#pragma unroll
        for (int u = 0; u < kLpBatch; ++u) {
          float s8 = 0.f, q8 = 0.f;  // (short sums first: a thread adds thousands)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float d = __builtin_fmaf(v[u].get(e), kLpLog2e, -base), p = __builtin_amdgcn_exp2f(d);
            s8 += p;
            q8 = __builtin_fmaf(p, fmaxf(d, kLpFloor2), q8);
          }
          s += s8;
          q += q8;
        }
        // the sums here: the compiler would take q's behind the alternatives, with all the terms they need
        if (TOP) asm volatile("" : "+v"(s), "+v"(q));
      }
      if constexpr (TOP) {
        const int batch = (c0 - first) / kLpRound + 1;
        if ((batch & (batch - 1)) == 0) {
          const uint32_t mine = reached(order_of(peak) >> 16, a.top < kLpWaves ? a.top : (a.top + kLpWaves - 1) / kLpWaves);
          if (lane == 0) put_shared(&reach[wave], mine);
        }
        if (c0 == first) __syncthreads();
        uint32_t all = get_shared(&reach[0]);
#pragma unroll
        for (int w = 1; w < kLpWaves; ++w) {
          const uint32_t other = get_shared(&reach[w]);
          all = (other < all) != (a.top < kLpWaves) ? other : all;
        }
        all = __builtin_amdgcn_readfirstlane(all);
        const u64 barrier = all ? ((u64)all << 48) - 1 : 0;
        limit = barrier > limit ? barrier : limit;
        // the least value with a key above the limit: of the limit's own value all entries from here on have lower keys
        // than those of a list that was cut down to it (a NaN above NaN and infinity: all pass, and keys decide)
        const float bar = limit ? value_of((uint32_t)(limit >> 32) + 1) : -INFINITY;
        const bool odd = !(s - s == 0.f);  // NaN or infinities among this thread's entries
        uint32_t bits = 0;                 // the entries of this thread's batch that reach the bar
#pragma unroll
        for (int u = 0; u < kLpBatch; ++u) {
          if (!__any(odd || !(high[u] < bar))) continue;
          v[u].again();
#pragma unroll
          for (int e = 0; e < 8; ++e) bits |= (v[u].get(e) < bar ? 0u : 1u) << (8 * u + e);
        }
        // an entry of each thread at a time, loaded again: the place of a vector's element is no register's name
        while (__any(bits != 0)) {
          const int which = bits ? __builtin_ctz(bits) : 0, at = c + (which >> 3) * (8 * kLpThreads) + (which & 7);
          const bool here = bits != 0 && at < end;
          bits &= bits - 1;
          const u64 key = here ? key_of(LpVec<ZT>::one(z + at), at) : 0;
          u64 take = __ballot(key > limit);
          if (count + __builtin_popcountll(take) > kLpList) {
            const u64 last = cut_list(lists[wave], count, a.top);
            limit = uniform_u64(last > limit ? last : limit);
            take = __ballot(key > limit);
          }
          if (key > limit) lists[wave][count + __builtin_popcountll(take & ((u64(1) << lane) - 1))] = key;
          count += __builtin_popcountll(take);
        }
      }
    }
    float most = peak;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
    if (most == -INFINITY) {
      m = -INFINITY;  // (and s is 0, or NaN)
    } else if (fabsf(most) <= kLpNear) {
      // against m itself, and q in units of e
      const float off = __builtin_fmaf(m, kLpLog2e, -base), f = __builtin_amdgcn_exp2f(-off);
      q = __builtin_fmaf(-off, s, q) * (f * kLpLn2);
      s *= f;
    } else {
      // this wave's entries again, against their largest: the products with log2 e are too coarse, or not finite
      m = most, s = q = 0.f;
      for (int c0 = first; c0 < end; c0 += kLpRound)
        for (int i = 0; i < 8 * kLpBatch; ++i) {
          const int at = c0 + 8 * (int)threadIdx.x + (i >> 3) * (8 * kLpThreads) + (i & 7);
          if (at >= end) continue;
          const float d = LpVec<ZT>::one(z + at) - m, p = lp_exp(d);
          s += p;
          q = __builtin_fmaf(p, fmaxf(d, kLpFloor), q);
        }
    }
    // the lanes' sums, then the waves'
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
      join_sums(m, s, q, __shfl_xor(m, off, 64), __shfl_xor(s, off, 64), __shfl_xor(q, off, 64));
    if (lane == 0) {
      sums[wave] = f32x4_t{m, s, q, 0.f};
      counts[wave] = count;
    }
    __syncthreads();
    if (TOP || wave == 0) {
      // (in one order in every wave)
      m = sums[0].x, s = sums[0].y, q = sums[0].z;
#pragma unroll
      for (int w = 1; w < kLpWaves; ++w) join_sums(m, s, q, sums[w].x, sums[w].y, sums[w].z);
      if (threadIdx.x == 0) {
        if (a.parts == 1) finish_row(a, row, y, zy, m, s, q);
        else a.sums[job] = f32x4_t{m, s, q, 0.f};
      }
    }
    if constexpr (TOP) {
#pragma unroll 1
      for (int i = threadIdx.x; i < kLpWaves * kLpList; i += kLpThreads) {
        if (i % kLpList >= counts[i / kLpList]) continue;
        const u64 key = lists[i / kLpList][i % kLpList];
        int place = 0;
#pragma unroll 1
        for (int w = 0; w < kLpWaves; ++w) place += place_of(key, lists[w], counts[w]);
        if (place >= a.top) continue;
        if (a.parts == 1) put_alternative(a, row, place, key, m, s);
        else a.keys[job * a.top + place] = key;
      }
      // a part of fewer entries than `top` fills up with keys below all others
      if (a.parts > 1) {
        int all = 0;
        for (int w = 0; w < kLpWaves; ++w) all += counts[w];
        for (int i = all + (int)threadIdx.x; i < a.top; i += kLpThreads) a.keys[job * a.top + i] = 0;
      }
    }
    __syncthreads();  // before the next row's sums and lists
  }
}

// Joins a row's parts: a workgroup per row. The parts' lists are in descending order, so `top`
// keys reach the least of their ceil(top / parts)th ones, and the largest of their last: only keys that
// reach both are ranked, about twice `top` of them.
template <typename ZT, bool TOP>
__global__ __launch_bounds__(kLpJoinThreads) void lp_join_kernel(LpArgs a) {
  __shared__ __attribute__((aligned(16))) u64 list[TOP ? kLpMaxParts * kLpMaxTop : 1];
  __shared__ int kept;
  const int lane = threadIdx.x & 63;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    int64_t y = -1;
    float zy = 0.f;
    if (threadIdx.x == 0 && a.tokens) {
      y = a.tokens[row];
      zy = token_logit<ZT>(a, row, y);
    }
    float m = -INFINITY, s = 0.f, q = 0.f;
    if (lane < a.parts) {
      const f32x4_t x = a.sums[row * a.parts + lane];
      m = x.x, s = x.y, q = x.z;
    }
    u64 bar = ~u64(0), last = 0;
    const u64* keys = a.keys + row * a.parts * a.top;
    if constexpr (TOP) {
      if (lane < a.parts) {
        bar = keys[lane * a.top + (a.top + a.parts - 1) / a.parts - 1];
        last = keys[lane * a.top + a.top - 1];
      }
      if (threadIdx.x == 0) kept = 0;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      join_sums(m, s, q, __shfl_xor(m, off, 64), __shfl_xor(s, off, 64), __shfl_xor(q, off, 64));
      if constexpr (TOP) {
        const u64 b1 = __shfl_xor(bar, off, 64), l1 = __shfl_xor(last, off, 64);
        bar = b1 < bar ? b1 : bar, last = l1 > last ? l1 : last;
      }
    }
    if (threadIdx.x == 0) finish_row(a, row, y, zy, m, s, q);
    if constexpr (TOP) {
      bar = last > bar ? last : bar;
      __syncthreads();
      for (int i = threadIdx.x; i < a.parts * a.top; i += kLpJoinThreads) {
        const u64 key = keys[i];
        if (key != 0 && key >= bar) list[atomicAdd(&kept, 1)] = key;
      }
      __syncthreads();
      const int count = kept;
      for (int i = threadIdx.x; i < count; i += kLpJoinThreads) {
        const u64 key = list[i];
        const int place = place_of(key, list, count);
        if (place < a.top) put_alternative(a, row, place, key, m, s);
      }
      __syncthreads();
    }
  }
}

// What the entries of a row need for their gradients.
struct LpRow {
  float base, ls;  // z - base - ls is the log probability
  float gl, flat, slope;
  int64_t y;
  bool live;
};

// A batch of a row's gradients, from entry c0 on.
template <typename ZT>
__device__ __forceinline__ void backward_batch(const ZT* z, ZT* dz, int V, int c0, const LpRow& r) {
  const int c = c0 + 8 * (int)threadIdx.x;
  LpVec<ZT> v[kLpBatch];
#pragma unroll
  for (int u = 0; u < kLpBatch; ++u) {
    const int at = c + u * (8 * kLpThreads);
    v[u].none();
    if (r.live && at + 8 <= V) v[u].load(z + at);
    else if (r.live && at < V) v[u].load_some(z + at, V - at);
  }
#pragma unroll
  for (int u = 0; u < kLpBatch; ++u) {
    const int at = c + u * (8 * kLpThreads);
    if (at >= V) continue;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = v[u].get(e) - r.base - r.ls;
      f[e] = lp_exp(d) * __builtin_fmaf(r.slope, fmaxf(d, kLpFloor), r.flat);
      if (at + e == r.y) f[e] += r.gl;
      if (!r.live) f[e] = 0.f;
    }
    if (at + 8 <= V) {
      LpVec<ZT>::store(dz + at, f);
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (at + e < V) LpVec<ZT>::put(dz + at + e, f[e]);
    }
  }
}

template <typename ZT>
__global__ __launch_bounds__(kLpThreads) void lp_backward_kernel(LpArgs a) {
  __shared__ float2 sums[kLpWaves];
  const int64_t parts = (a.V + kLpRound - 1) / kLpRound, jobs = a.rows * parts;
  for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
    const int64_t row = job / parts;
    const int c0 = (int)(job - row * parts) * kLpRound;
    const ZT* z = static_cast<const ZT*>(a.z) + row * a.ldz;
    ZT* dz = static_cast<ZT*>(a.dz) + row * a.lddz;
    LpRow r;
    r.y = a.tokens[row];
    r.base = a.lse[row], r.ls = 0.f;
    r.live = r.y >= 0 && r.y < a.V && r.base != -INFINITY;
    const float ge = a.grad_entropy ? a.grad_entropy[row] : 0.f;
    r.gl = a.grad_logp ? a.grad_logp[row] : 0.f;
    r.flat = ge != 0.f ? -__builtin_fmaf(ge, a.entropy[row], r.gl) : -r.gl, r.slope = -ge;
    if (!(r.live && fabsf(r.base) >= kLpFar && r.base != INFINITY)) {
      backward_batch(z, dz, a.V, c0, r);
      continue;
    }
    // a far row is one workgroup's (dz may be z: nobody else may write it before it is read)
    if (c0 > 0) continue;
    float m = -INFINITY, s = 0.f, q = 0.f;
    for (int at = threadIdx.x; at < a.V; at += kLpThreads) m = fmaxf(m, LpVec<ZT>::one(z + at));
    for (int at = threadIdx.x; at < a.V; at += kLpThreads) s += lp_exp(LpVec<ZT>::one(z + at) - (m == -INFINITY ? 0.f : m));
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) join_sums(m, s, q, __shfl_xor(m, off, 64), __shfl_xor(s, off, 64), 0.f);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = make_float2(m, s);
    __syncthreads();
    m = -INFINITY, s = 0.f;
#pragma unroll
    for (int w = 0; w < kLpWaves; ++w) join_sums(m, s, q, sums[w].x, sums[w].y, 0.f);
    r.base = m, r.ls = logf(s);
    for (int at = 0; at < a.V; at += kLpRound) backward_batch(z, dz, a.V, at, r);
    __syncthreads();  // before the next far row's sums
  }
}

size_t elem(rgc_dtype_t t) { return t == RGC_F32 ? 4 : 2; }

// Parts of a row of the forward: one where the rows give each compute unit more than three
// workgroups, else as many as give it six, its fill of waves, of at least half a batch each
// (their join is a launch of 5 us). bf16, eight alternatives, against four of
// them: 150 x 131072 26 and 24 us, 300 x 131072 36 and 34, 1003 x 50021 in one part 37 either way
// and 51 in three.
int64_t parts_of(int64_t rows, int64_t V) {
  const int64_t want = ((int64_t)device_compute_units() * 6) / rows;
  const int64_t most = (V + kLpRound / 2 - 1) / (kLpRound / 2);
  int64_t parts = want < most ? want : most;
  if (parts > kLpMaxParts) parts = kLpMaxParts;
  return parts < 1 ? 1 : parts;
}
int64_t part_of(int64_t V, int64_t parts) { return ((V + parts - 1) / parts + 7) / 8 * 8; }

size_t sums_bytes(int64_t rows, int64_t parts) { return ((size_t)rows * parts * sizeof(f32x4_t) + 255) / 256 * 256; }

rgc_status_t check_shape(rgc_dtype_t zt, int64_t rows, int64_t V, int64_t top) {
  if (zt != RGC_BF16 && zt != RGC_F32) return RGC_ERR_UNSUPPORTED;
  if (rows < 0 || V <= 0 || top < 0 || top > V) return RGC_ERR_SHAPE;
  if (rows > kLpMaxRows || V > kLpMaxVocab || top > kLpMaxTop) return RGC_ERR_UNSUPPORTED;
  return RGC_OK;
}
rgc_status_t check_rows(const void* p, int64_t ld, int64_t V, rgc_dtype_t t) {
  if (!p) return RGC_ERR_NULL;
  if (ld < V) return RGC_ERR_SHAPE;
  if (ld > kLpMaxLeadingDim) return RGC_ERR_UNSUPPORTED;
  if (!aligned_to(p, elem(t))) return RGC_ERR_ALIGN;
  return RGC_OK;
}

unsigned grid_of(int64_t jobs) {
  const int64_t most = int64_t(1) << 20;  // (launches stay below 2^31 threads)
  return (unsigned)(jobs < most ? jobs : most);
}

template <typename ZT, bool TOP>
rgc_status_t forward_launch(const LpArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((lp_forward_kernel<ZT, TOP>), dim3(grid_of(a.rows * a.parts)), dim3(kLpThreads), 0, s, a);
  if (a.parts > 1) hipLaunchKernelGGL((lp_join_kernel<ZT, TOP>), dim3(grid_of(a.rows)), dim3(TOP ? kLpJoinThreads : 64), 0, s, a);
  return hipGetLastError() == hipSuccess ? RGC_OK : RGC_ERR_HIP;
}

}  // namespace
}  // namespace rgc

using namespace rgc;

extern "C" size_t rgc_log_prob_forward_workspace_size(int64_t rows, int64_t V, int64_t top) {
  if (check_shape(RGC_BF16, rows, V, top) != RGC_OK || rows == 0) return 0;
  const int64_t parts = parts_of(rows, V);
  return parts == 1 ? 0 : sums_bytes(rows, parts) + (size_t)(rows * parts * top) * sizeof(u64);
}

extern "C" rgc_status_t rgc_log_prob_forward(rgc_dtype_t zt, const void* Z, int64_t ldz, const int64_t* tokens, float* logp,
                                             float* entropy, float* lse, int64_t top, float* top_logp, int64_t* top_ids,
                                             int64_t rows, int64_t V, void* ws, size_t ws_bytes, void* stream) {
  rgc_status_t st = check_shape(zt, rows, V, top);
  if (st != RGC_OK || rows == 0) return st;
  if ((st = check_rows(Z, ldz, V, zt)) != RGC_OK) return st;
  if (!entropy || !lse || (tokens && !logp) || (top > 0 && (!top_logp || !top_ids))) return RGC_ERR_NULL;
  if (!aligned_to(tokens, 8) || !aligned_to(logp, 4) || !aligned_to(entropy, 4) || !aligned_to(lse, 4) ||
      !aligned_to(top_logp, 4) || !aligned_to(top_ids, 8))
    return RGC_ERR_ALIGN;
  const size_t need = rgc_log_prob_forward_workspace_size(rows, V, top);
  if (need > 0 && (!ws || ws_bytes < need)) return RGC_ERR_WORKSPACE;
  if (!aligned_to(ws, 256)) return RGC_ERR_ALIGN;
  LpArgs a{};
  a.z = Z, a.ldz = ldz, a.rows = rows, a.V = (int)V, a.top = (int)top;
  a.parts = (int)parts_of(rows, V), a.part = (int)part_of(V, a.parts);
  a.tokens = tokens, a.logp = logp, a.entropy = entropy, a.lse = lse, a.top_logp = top_logp, a.top_ids = top_ids;
  if (a.parts > 1) {
    a.sums = static_cast<f32x4_t*>(ws);
    a.keys = reinterpret_cast<u64*>(static_cast<char*>(ws) + sums_bytes(rows, a.parts));
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (zt == RGC_F32) return top > 0 ? forward_launch<float, true>(a, s) : forward_launch<float, false>(a, s);
  return top > 0 ? forward_launch<uint16_t, true>(a, s) : forward_launch<uint16_t, false>(a, s);
}

extern "C" rgc_status_t rgc_log_prob_backward(rgc_dtype_t zt, const void* Z, int64_t ldz, const int64_t* tokens,
                                              const float* lse, const float* entropy, const float* grad_logp,
                                              const float* grad_entropy, void* dZ, int64_t lddz, int64_t rows, int64_t V,
                                              void* stream) {
  rgc_status_t st = check_shape(zt, rows, V, 0);
  if (st != RGC_OK || rows == 0) return st;
  if ((st = check_rows(Z, ldz, V, zt)) != RGC_OK) return st;
  if ((st = check_rows(dZ, lddz, V, zt)) != RGC_OK) return st;
  if (!tokens || !lse || (!grad_logp && !grad_entropy) || (grad_entropy && !entropy)) return RGC_ERR_NULL;
  if (!aligned_to(tokens, 8) || !aligned_to(lse, 4) || !aligned_to(entropy, 4) || !aligned_to(grad_logp, 4) ||
      !aligned_to(grad_entropy, 4))
    return RGC_ERR_ALIGN;
  LpArgs a{};
  a.z = Z, a.ldz = ldz, a.rows = rows, a.V = (int)V, a.tokens = tokens, a.dz = dZ, a.lddz = lddz;
  a.lse = const_cast<float*>(lse), a.entropy = const_cast<float*>(entropy);
  a.grad_logp = grad_logp, a.grad_entropy = grad_entropy;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const unsigned grid = grid_of(rows * ((V + kLpRound - 1) / kLpRound));
  if (zt == RGC_F32) hipLaunchKernelGGL(lp_backward_kernel<float>, dim3(grid), dim3(kLpThreads), 0, s, a);
  else hipLaunchKernelGGL(lp_backward_kernel<uint16_t>, dim3(grid), dim3(kLpThreads), 0, s, a);
  return hipGetLastError() == hipSuccess ? RGC_OK : RGC_ERR_HIP;
}
