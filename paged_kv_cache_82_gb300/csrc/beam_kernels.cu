// beam_kernels.cu -- the best continuations of each group of beams
// (pa_beam_select).
//
//   score(w, t) = beam_scores[w] + x[w][t] - log sum_u exp(x[w][u])
//   the K largest over the W beams and V tokens of a group
//
// Each logit is read once.  A CTA takes a chunk of a row into registers and
// leaves the chunk's maximum m, its sum of exp(x - m) and its K largest logits;
// a second kernel, a CTA to a group, joins the sums of each row (the running
// maximum of an online softmax, over chunks) and picks K of the W x chunks x K
// candidates.
//
// The K largest of a chunk without sorting it: eight warps, each with its q-th
// largest lane maximum, q = ceil(K / 8); the smallest of these eight numbers is
// a threshold that at least 8 q >= K logits reach, and about 20 of 16384 do for K
// = 8.  Those go to a list in shared memory, where each counts the larger ones.
// (Where some lanes or warps hold most of the largest logits, as in a vocabulary
// sorted by frequency, the same again over what reached the threshold: the case
// below with a falling trend 22 us with it, 33 without, sorted 36 and 243.)
//
// Which tokens come back must not depend on the rounding of fp32 sums: scores are
// compared in 64 bits, and where two beams' scores lie closer than the fp32 sums
// resolve (kNear), the sums of those rows are taken again with exponentials in
// two fp32 parts and the group is picked again (about one group in 2000 of
// unlike beams with K = 4, one in 100 with K = 64, always for beams that are copies of
// each other).  In 64 groups of 4 beams of 128256 bf16 logits that takes 36 us more
// for one pair of such beams, 85 where all beams are copies.
//
// 64 groups of 4 beams of 128256 bf16 logits, a tenth of them finished, 59 MB: 22.0 us,
// where reading them at a plain copy's rate takes 8.7 (other logits in each call, more in
// all than the L2 holds; 20.5 where it holds them).  The chunks alone take 16 (3.7 TB/s):
// half of the issue slots (nine instructions to a logit), the rest waiting for loads and for
// the other warps of a CTA, four CTAs to an SM.  The join adds 6, a chain of short steps.
// 32 groups of 8 beams of 50257 fp32 logits 22.1 us, 15 of them the chunks; one group of 4
// beams of 32000 7.5 us.
#include <cooperative_groups.h>
#include <float.h>
#include <math.h>

#include "pa_beam.h"
#include "pa_common.cuh"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kWarps = kBeamThreads / 32;
constexpr int kVecCap = 512;    // 16-byte vectors of a chunk that hold a candidate
constexpr int kListCap = 1024;  // candidates of a chunk, and of a group
constexpr int kMaxJoinCtas = 4;
constexpr int kBatch = 8;
constexpr float kLog2e = 1.44269502162933349609375f;  // off by less than 2^-25 of itself
constexpr float kMasked = -1e30f;  // the lowest value of a type, or next to it
// Two scores' difference from which on the fp32 sums decide.  A row's log-sum is
// off by at most: 2^-22 (the exponential) + ln 2 x 2^-23 x the mean of |log2 p| over
// the row, below log2 V <= 24 (the exponent's rounding and log2 e's) + 18 x 2^-24 (8
// additions in a thread, 10 above) + 2 x 2^-22 (warps and chunks joined) = 3.8e-6.
constexpr double kNear = 1e-5;

// ---- order of logits ---------------------------------------------------------
// whole numbers in the order of the floats (-0 = 0)
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
  return b >> 63 ? ~b : b | (1ull << 63);
}
// a logit and its token: larger keys are better (equal logits: the lower token);
// 0: none
__device__ __forceinline__ uint64_t make_key(float x, int token) {
  return (uint64_t)ordered(x) << 32 | (uint32_t)~token;
}
// NaN counts as -inf, +inf as the largest number
__device__ __forceinline__ float clean(float x) {
  return fminf(fmaxf(x, -INFINITY), FLT_MAX);
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint64_t warp_max_u64(uint64_t v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const uint64_t o = __shfl_xor_sync(~0u, v, d);
    v = o > v ? o : v;
  }
  return v;
}

// This warp's q-th largest of its lanes' numbers (0 where there are fewer than
// q above 0).
__device__ __forceinline__ uint32_t warp_qth_largest(uint32_t v, int q) {
  uint32_t top = __reduce_max_sync(~0u, v);
  for (int i = 1; i < q && i < 32; ++i) {
    const unsigned who = __ballot_sync(~0u, v == top);
    if ((threadIdx.x & 31) == __ffs(who) - 1) v = 0;
    top = __reduce_max_sync(~0u, v);
  }
  return q > 32 ? 0 : top;
}

// ---- elements of a 16-byte load ------------------------------------------------
// get: one element; pair: elements 2 i and 2 i + 1; Max: the largest of what it has
// been given, NaN passed over
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
template <typename T>
struct Pack;
template <>
struct Pack<float> {
  static constexpr int kN = 4;
  static constexpr uint32_t kNegInf = 0xff800000u, kNegInfs = kNegInf;
  static constexpr float kLowest = -FLT_MAX;
  static __device__ __forceinline__ uint32_t bits(const float* p) { return __float_as_uint(*p); }
  static __device__ __forceinline__ float get(const float* p) { return *p; }
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    return __uint_as_float(word(v, i));
  }
  static __device__ __forceinline__ float2 pair(const uint4& v, int i) {
    return make_float2(get(v, 2 * i), get(v, 2 * i + 1));
  }
  struct Max {
    float m;
    __device__ __forceinline__ explicit Max(const uint4& v)
        : m(fmaxf(fmaxf(get(v, 0), get(v, 1)), fmaxf(get(v, 2), get(v, 3)))) {}
    __device__ __forceinline__ void add(const Max& o) { m = fmaxf(m, o.m); }
    __device__ __forceinline__ float value() const { return fmaxf(m, -INFINITY); }
    __device__ __forceinline__ bool reaches(float x) const { return m >= x; }
  };
};
template <>
struct Pack<__nv_bfloat16> {
  static constexpr int kN = 8;
  static constexpr uint32_t kNegInf = 0xff80u, kNegInfs = 0xff80ff80u;
  static constexpr float kLowest = -0x1.fep127f;
  static __device__ __forceinline__ uint32_t bits(const __nv_bfloat16* p) {
    return __bfloat16_as_ushort(*p);
  }
  static __device__ __forceinline__ float get(const __nv_bfloat16* p) {
    return __bfloat162float(*p);
  }
  static __device__ __forceinline__ float2 pair(const uint4& v, int i) {
    const uint32_t w = word(v, i);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    const float2 p = pair(v, i >> 1);
    return i & 1 ? p.y : p.x;
  }
  struct Max {
    __nv_bfloat162 m;
    __device__ __forceinline__ explicit Max(const uint4& v) {
      const auto* w = reinterpret_cast<const __nv_bfloat162*>(&v);
      m = __hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3]));
    }
    __device__ __forceinline__ void add(const Max& o) { m = __hmax2(m, o.m); }
    __device__ __forceinline__ float value() const {
      const float2 p = __bfloat1622float2(m);
      return fmaxf(fmaxf(p.x, p.y), -INFINITY);
    }
    __device__ __forceinline__ bool reaches(float x) const {
      return __hge2_mask(m, __float2bfloat162_rn(x)) != 0;
    }
  };
};
template <>
struct Pack<__half> {
  static constexpr int kN = 8;
  static constexpr uint32_t kNegInf = 0xfc00u, kNegInfs = 0xfc00fc00u;
  static constexpr float kLowest = -65504.f;
  static __device__ __forceinline__ uint32_t bits(const __half* p) { return __half_as_ushort(*p); }
  static __device__ __forceinline__ float get(const __half* p) { return __half2float(*p); }
  static __device__ __forceinline__ float2 pair(const uint4& v, int i) {
    const uint32_t w = word(v, i);
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    const float2 p = pair(v, i >> 1);
    return i & 1 ? p.y : p.x;
  }
  struct Max {
    __half2 m;
    __device__ __forceinline__ explicit Max(const uint4& v) {
      const auto* w = reinterpret_cast<const __half2*>(&v);
      m = __hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3]));
    }
    __device__ __forceinline__ void add(const Max& o) { m = __hmax2(m, o.m); }
    __device__ __forceinline__ float value() const {
      const float2 p = __half22float2(m);
      return fmaxf(fmaxf(p.x, p.y), -INFINITY);
    }
    __device__ __forceinline__ bool reaches(float x) const {
      return __hge2_mask(m, __float2half2_rn(x)) != 0;
    }
  };
};

// the elements [i0, i0 + kN) of a row of n where they are not all inside it: what lies
// outside is -inf and not read
template <typename T>
__device__ __noinline__ uint4 load_edge(const T* row, int i0, int n) {
  constexpr int kN = Pack<T>::kN, kPer = kN / 4;  // kPer: elements of a 32-bit word
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    w[k] = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int i = i0 + k * kPer + e;
      const uint32_t b = i >= 0 && i < n ? Pack<T>::bits(row + i) : Pack<T>::kNegInf;
      w[k] |= b << (e * 16);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// 16-byte aligned where whole
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, int i0, int n) {
  if (i0 >= 0 && i0 + Pack<T>::kN <= n) return __ldcs(reinterpret_cast<const uint4*>(row + i0));
  return load_edge<T>(row, i0, n);
}

struct BeamK {
  BeamArgs a;
  int chunks;
  unsigned stride;  // through a group's candidates
  uint64_t* keys;  // [rows][chunks][K], best first
  float2* stats;   // [rows][chunks]: maximum, sum of exp(x - maximum)
};

// The chunk's sum where the fast one's exponents overflowed (the logits read again).
template <typename T, int kVecs>
__device__ __noinline__ float odd_sum(const T* x, int base, int V, float mx) {
  using P = Pack<T>;
  float2 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int i = 0; i < kVecs; ++i) {
    const uint4 v = load_vec<T>(x, base + i * kBeamThreads * P::kN, V);
#pragma unroll
    for (int j = 0; j < P::kN / 2; ++j) {
      const float2 e = P::pair(v, j);
      acc[j & 3].x += exp2_approx((clean(e.x) - mx) * kLog2e);
      acc[j & 3].y += exp2_approx((clean(e.y) - mx) * kLog2e);
    }
  }
  return ((acc[0].x + acc[1].x) + (acc[2].x + acc[3].x)) +
         ((acc[0].y + acc[1].y) + (acc[2].y + acc[3].y));
}

// The K best of a list of n: each counts the better ones, up to K.
__device__ __forceinline__ void rank_list(const uint64_t* list, int n, int K, uint64_t* keys) {
  for (int i = threadIdx.x; i < n; i += kBeamThreads) {
    const uint64_t mine = list[i];
    int rank = 0;
    for (int j = 0; j < n && rank < K; j += 4)
#pragma unroll
      for (int k = 0; k < 4; ++k) rank += j + k < n && list[j + k] > mine;
    if (rank < K) keys[rank] = mine;
  }
  for (int i = n + threadIdx.x; i < K; i += kBeamThreads) keys[i] = 0;
}

// More vectors reach the threshold than K should leave: the logits of some lanes or warps lie
// above the others' (a vocabulary sorted by frequency).  The threshold once more, of the
// vectors kept, dealt out over all warps.
template <typename T>
__device__ __noinline__ float tighten(const uint4* vecs, int n, int K, uint32_t* s_bar,
                                      float floor_x) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float m = -INFINITY;
#pragma unroll 1
  for (int i = lane * kWarps + warp; i < n; i += kBeamThreads)
    m = fmaxf(m, (typename Pack<T>::Max(vecs[i])).value());
  const uint32_t bar = warp_qth_largest(ordered(fminf(m, FLT_MAX)), (K + kWarps - 1) / kWarps);
  __syncthreads();  // (s_bar has been read)
  if (lane == 0) s_bar[warp] = bar;
  __syncthreads();
  return fmaxf(unordered(__reduce_min_sync(~0u, s_bar[lane & (kWarps - 1)])), floor_x);
}

// More logits than there is room for reach the threshold: those of a chunk of equal ones
// (masked by a type's lowest value, say), as a rule.  The logits above it to the list, and
// then of the equal ones the first; where even the former are too many, above a threshold
// of the vectors kept; and where that does not help, the best key below the last one taken,
// K times.
template <typename T, int kVecs>
__device__ __noinline__ void pick_from_many(const T* x, int base, int V, int K, float floor_x,
                                            const uint4* vecs, int kept, uint64_t* list,
                                            int* s_count, int* warp_sums, uint32_t* s_bar,
                                            uint64_t* s_best, uint64_t* keys) {
  using P = Pack<T>;
  constexpr int kStep = kBeamThreads * P::kN;
  int n;
#pragma unroll 1
  for (bool again = true;; again = false) {
    __syncthreads();
    if (threadIdx.x == 0) *s_count = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < kVecs; ++i) {
      const int at = base + i * kStep;
      const uint4 v = load_vec<T>(x, at, V);
#pragma unroll
      for (int j = 0; j < P::kN; ++j) {
        const float e = clean(P::get(v, j));
        if (e > floor_x) {
          const int place = atomicAdd(s_count, 1);
          if (place < kListCap) list[place] = make_key(e, at + j);
        }
      }
    }
    __syncthreads();
    n = *s_count;
    if (n <= kListCap || !again) break;
    const float higher = tighten<T>(vecs, kept, K, s_bar, floor_x);
    if (higher == floor_x) break;
    floor_x = higher;
  }
  if (n <= kListCap) {
#pragma unroll 1
    for (int i = 0; i < kVecs && n < K; ++i) {
      const int at = base + i * kStep;
      const uint4 v = load_vec<T>(x, at, V);
      int equal = 0, total;
#pragma unroll
      for (int j = 0; j < P::kN; ++j) equal += clean(P::get(v, j)) == floor_x;
      int place = n + block_scan_excl(equal, warp_sums + kWarps, warp_sums);
      total = warp_sums[kWarps];
#pragma unroll
      for (int j = 0; j < P::kN; ++j)
        if (clean(P::get(v, j)) == floor_x) {
          if (place < K) list[place] = make_key(floor_x, at + j);
          ++place;
        }
      n = min(n + total, max(n, K));
      __syncthreads();  // the scan's memory is written again; the list is complete
    }
    rank_list(list, n, K, keys);
    return;
  }
  uint64_t last = ~0ull;
  for (int k = 0; k < K; ++k) {
    uint64_t best = 0;
#pragma unroll 1
    for (int i = 0; i < kVecs; ++i) {
      const int at = base + i * kStep;
      const uint4 v = load_vec<T>(x, at, V);
#pragma unroll
      for (int j = 0; j < P::kN; ++j) {
        const float e = P::get(v, j);
        const uint64_t key = make_key(fminf(e, FLT_MAX), at + j);
        if (e > -INFINITY && key < last && key > best) best = key;
      }
    }
    best = warp_max_u64(best);
    if ((threadIdx.x & 31) == 0) s_best[threadIdx.x >> 5] = best;
    __syncthreads();
    best = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) best = s_best[w] > best ? s_best[w] : best;
    __syncthreads();
    if (threadIdx.x == 0) keys[k] = best;
    last = best;
  }
}

// One chunk of one row.
template <typename T, int kVecs>
__global__ void __launch_bounds__(kBeamThreads, kVecs >= 8 ? 4 : 5)
    beam_chunk_kernel(BeamK p) {
  using P = Pack<T>;
  constexpr int kN = P::kN, kStep = kBeamThreads * kN;
  __shared__ uint4 vecs[kVecCap];
  __shared__ int vec_at[kVecCap];
  __shared__ uint64_t list[kListCap];
  __shared__ uint32_t s_max[kWarps], s_bar[kWarps];
  __shared__ float s_sum[kWarps];
  __shared__ uint64_t s_best[kWarps];
  __shared__ int s_count, s_vecs, s_scan[kWarps + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / (unsigned)p.chunks;
  const int chunk = (int)(blockIdx.x - row * p.chunks);
  const int K = p.a.num_selected, V = p.a.vocab_size;
  pdl_launch_dependents();
  if (p.a.finished && p.a.finished[row]) return;  // (its logits are not looked at)
  const T* x = static_cast<const T*>(p.a.logits) + row * p.a.row_stride;
  // the row seen from the 16-byte boundary at or before its start
  const int first = chunk * (kVecs * kStep) -
                    (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const int base = first + tid * kN;
  uint4 v[kVecs];
  if (first >= 0 && first + kVecs * kStep <= V) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      v[i] = __ldcs(reinterpret_cast<const uint4*>(x + base + i * kStep));
  } else {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int at = base + i * kStep;
      v[i] = make_uint4(P::kNegInfs, P::kNegInfs, P::kNegInfs, P::kNegInfs);
      if (at >= 0 && at + kN <= V) v[i] = __ldcs(reinterpret_cast<const uint4*>(x + at));
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {  // the vector that a row's start or end cuts
      const int at = base + i * kStep;
      if ((at < 0 && at + kN > 0) || (at < V && at + kN > V)) v[i] = load_edge<T>(x, at, V);
    }
  }
  typename P::Max tops(v[0]);
#pragma unroll
  for (int i = 1; i < kVecs; ++i) tops.add(typename P::Max(v[i]));
  const float m = fminf(tops.value(), FLT_MAX);
  const uint32_t om = ordered(m);
  // (at least q lanes of each warp reach the q-th largest: 8 q logits of the CTA)
  const int q = (K + kWarps - 1) / kWarps;
  const uint32_t wmax = __reduce_max_sync(~0u, om);
  const uint32_t bar = q == 1 ? wmax : warp_qth_largest(om, q);
  // ---- sum of 2^(x h - c), h = fl32(log2 e), c = fl32(m h) for the warp's maximum m.  x h
  // - c is (x - m) h, one rounding, and m h - c, which is exact in fp32 and comes off at
  // the end; h's error counts for x - m only.  (No barrier before it: a warp whose logits
  // are there goes on.  One whose logits are all masked by a type's lowest value sums 0.)
  const float wm = unordered(wmax);
  const float c = wm > kMasked ? wm * kLog2e : 0.f;
  float2 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float2(0.f, 0.f);
  const float2 h2 = make_float2(kLog2e, kLog2e), c2 = make_float2(-c, -c);
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int j = 0; j < kN / 2; ++j) {
      const float2 e = P::pair(v[i], j);
      const float2 y = __ffma2_rn(e, h2, c2);
      acc[j & 3] = __fadd2_rn(acc[j & 3], make_float2(exp2_approx(y.x), exp2_approx(y.y)));
    }
  const float2 a01 = __fadd2_rn(acc[0], acc[1]), a23 = __fadd2_rn(acc[2], acc[3]);
  const float2 a03 = __fadd2_rn(a01, a23);
  float sum = a03.x + a03.y;
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  if (lane == 0) {
    s_max[warp] = wmax;
    s_bar[warp] = bar;
    s_sum[warp] = sum;
  }
  if (tid == 0) s_count = s_vecs = 0;
  __syncthreads();
  const uint32_t omax = __reduce_max_sync(~0u, s_max[lane & (kWarps - 1)]);
  const uint32_t least = __reduce_min_sync(~0u, s_bar[lane & (kWarps - 1)]);
  const float mx = unordered(omax);
  const int64_t out = row * p.chunks + chunk;
  if (mx == -INFINITY) {  // nothing here (uniform over the CTA)
    if (tid == 0) p.stats[out] = make_float2(-INFINITY, 0.f);
    for (int i = tid; i < K; i += kBeamThreads) p.keys[out * K + i] = 0;
    return;
  }
  // ---- the vectors that hold a logit at or above the threshold, to shared memory
  float floor_x = fmaxf(unordered(least), P::kLowest);
  unsigned hits = 0;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) hits |= (typename P::Max(v[i])).reaches(floor_x) ? 1u << i : 0u;
  if (hits) {
    int at = atomicAdd(&s_vecs, __popc(hits));
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (hits >> i & 1) {
        if (at < kVecCap) {
          vecs[at] = v[i];
          vec_at[at] = base + i * kStep;
        }
        ++at;
      }
  }
  // ---- the warps' sums, all relative to the largest maximum
  {
    const float w = unordered(s_max[lane & (kWarps - 1)]);
    const float d = fmaf(w, kLog2e, -(w * kLog2e));
    sum = w > kMasked ? s_sum[lane & (kWarps - 1)] * exp2f((w - mx) * kLog2e - d) : 0.f;
  }
#pragma unroll
  for (int d = kWarps / 2; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  __syncthreads();
  const int n_vecs = s_vecs;
  if (n_vecs > 2 * K + 64 && n_vecs <= kVecCap)  // (some K to 2 K are usual)
    floor_x = tighten<T>(vecs, n_vecs, K, s_bar, floor_x);
  if (n_vecs <= kVecCap)  // the logits among theirs
    for (int e = tid; e < n_vecs * kN; e += kBeamThreads) {
      const int at = vec_at[e / kN] + e % kN;
      const float f = P::get(reinterpret_cast<const T*>(vecs) + e);
      if (f >= floor_x) {
        const int n = atomicAdd(&s_count, 1);
        if (n < kListCap) list[n] = make_key(fminf(f, FLT_MAX), at);
      }
    }
  // NaN, infinite or huge logits: the exponents above overflowed.  (Uniform.)
  const bool odd = !(sum >= 0.5f && sum < INFINITY) || fabsf(mx) > 1e6f;
  if (odd) {
    float t = odd_sum<T, kVecs>(x, base, V, mx);
#pragma unroll
    for (int d = 16; d; d >>= 1) t += __shfl_xor_sync(~0u, t, d);
    __syncthreads();
    if (lane == 0) s_sum[warp] = t;
    __syncthreads();
    sum = s_sum[lane & (kWarps - 1)];
#pragma unroll
    for (int d = kWarps / 2; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  }
  if (tid == 0) p.stats[out] = make_float2(mx, sum);
  uint64_t* keys = p.keys + out * K;
  __syncthreads();
  const int n = n_vecs <= kVecCap ? s_count : kListCap + 1;
  if (n <= kListCap)
    rank_list(list, n, K, keys);
  else
    pick_from_many<T, kVecs>(x, base, V, K, floor_x, vecs, min(n_vecs, kVecCap), list, &s_count,
                             s_scan, s_bar, s_best, keys);
}

// ---- sums again, in two fp32 parts ---------------------------------------------
// exp(t) for t in [-60, 0]: t = (64 n + j) ln 2 / 64 + r, exp = 2^n 2^(j/64) e^r
// (P. T. P. Tang, "Table-Driven Implementation of the Exponential Function", ACM
// TOMS 15, 1989).  ln 2 / 64 in three parts, the first two of 11 bits, so that
// their products with 64 n + j (13 bits) and the differences from t are exact.
constexpr double kLn2By64 = 0.010830424696249145;  // ln 2 / 64
constexpr float kC1 = (float)((long long)(kLn2By64 * 131072.0) / 131072.0);  // to 2^-17
constexpr float kC2 =
    (float)((long long)((kLn2By64 - (double)kC1) * 268435456.0) / 268435456.0);  // to 2^-28
constexpr float kC3 = (float)(kLn2By64 - (double)kC1 - (double)kC2);

struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float a, float b) {  // a + b, |b| small
    const float s = hi + a, z = s - hi;
    lo += ((hi - (s - z)) + (a - z)) + b;
    hi = s;
  }
};

__device__ __forceinline__ void add_exp(Sum2& acc, float x, float mx, const float2* table) {
  // t + t_lo = x - mx exactly
  const float t = x - mx, z = t - x;
  if (!(t >= -60.f)) return;  // (below 2^-86 of the largest term; NaN and -inf too)
  const float t_lo = (x - (t - z)) - (mx + z);
  const float kf = rintf(t * (float)(1.0 / kLn2By64));
  const int k = (int)kf;
  const float r2 = fmaf(-kf, kC2, fmaf(-kf, kC1, t));
  const float p3 = kf * kC3;
  const float r = r2 - p3;
  const float r_lo = ((r2 - r) - p3) + t_lo;
  // e^r - 1 = r + q, |r| < 2^-7.5
  const float q = fmaf(r * r, fmaf(r, fmaf(r, 1.f / 24, 1.f / 6), 0.5f), r_lo);
  const float2 w = table[k & 63];
  const float a = w.x * r, a_lo = fmaf(w.x, r, -a);
  const float s = w.x + a;
  const float s_lo = ((w.x - s) + a) + (a_lo + fmaf(w.x, q, fmaf(w.y, r, w.y)));
  const float scale = __int_as_float((127 + (k >> 6)) << 23);
  acc.add(s * scale, s_lo * scale);
}

// How a row's vectors of kN logits, counted from its first one, can be loaded
enum RowStart {
  kOnVectors,  // it starts on 16 bytes: a load to a vector
  kOnWords,    // on 4: four loads
  kInWords,    // on 2: five, of which the vector is the inner halves
};

// The kN logits from i on (i < n) of a row of n, what lies past its end being -inf; kInWords:
// those from i - 1 on and, in `fifth`, two more.
template <typename T, int kStart>
__device__ __forceinline__ uint4 load_from(const T* row, int i, int n, uint32_t& fifth) {
  constexpr int kN = Pack<T>::kN;
  if constexpr (kStart == kOnVectors) return load_vec<T>(row, i, n);
  if constexpr (kStart == kInWords) --i;
  if (i >= 0 && i + kN + (kStart == kInWords ? 2 : 0) <= n) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(row + i);
    if constexpr (kStart == kInWords) fifth = __ldg(w + 4);
    return make_uint4(__ldg(w), __ldg(w + 1), __ldg(w + 2), __ldg(w + 3));
  }
  if constexpr (kStart == kInWords) fifth = load_edge<T>(row, i + kN, n).x;
  return load_edge<T>(row, i, n);
}

// A thread's part of a row: vectors first, first + step, ..., kAhead at a time with as many on
// their way.  They are counted from the row's first logit, wherever in 16 bytes it lies:
// which logits are added in which order must not depend on that, or beams that are copies
// of each other would have sums that differ in their last bits.  (Words one after another
// in a loop: few instructions to fetch for code that is rarely run.)
template <typename T, int kStart>
__device__ __noinline__ double sum_from(const T* x, int V, float mx, const float2* table,
                                        int first, int step) {
  using P = Pack<T>;
  // (Fewer where a fifth word takes registers: with four the join saves more of its own
  // around the call, 0.6 us of every selection.  64 groups of 4 copies of 128255 bf16 logits
  // 106.4 us with two, 108.4 with three; of 128256, all on vectors, 105.7.)
  constexpr int kAhead = kStart == kInWords ? 2 : 4;
  const uint4 none = make_uint4(P::kNegInfs, P::kNegInfs, P::kNegInfs, P::kNegInfs);
  Sum2 acc[2];
  int i = first * P::kN;
  const int hop = step * P::kN;
  uint4 next[kAhead];
  uint32_t fifth[kAhead];
  auto fetch = [&] {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      fifth[u] = P::kNegInfs;
      next[u] = i + u * hop < V ? load_from<T, kStart>(x, i + u * hop, V, fifth[u]) : none;
    }
  };
  fetch();
#pragma unroll 1
  while (i < V) {
    uint4 v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      v[u] = next[u];
      if (kStart == kInWords)
        v[u] = make_uint4(__funnelshift_r(v[u].x, v[u].y, 16), __funnelshift_r(v[u].y, v[u].z, 16),
                          __funnelshift_r(v[u].z, v[u].w, 16),
                          __funnelshift_r(v[u].w, fifth[u], 16));
    }
    i += kAhead * hop;
    fetch();
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int j = 0; j < P::kN / 4; ++j)
          add_exp(acc[j & 1], clean(P::get(v[u], j)), mx, table);
        v[u] = make_uint4(v[u].y, v[u].z, v[u].w, v[u].x);
      }
  }
  return ((double)acc[0].hi + (double)acc[1].hi) + ((double)acc[0].lo + (double)acc[1].lo);
}

template <typename T>
__device__ __forceinline__ double precise_sum(const void* logits, int64_t at, int V, float mx,
                                              const float2* table, int first, int step) {
  const T* x = static_cast<const T*>(logits) + at;
  const unsigned start = (unsigned)(reinterpret_cast<uintptr_t>(x) & 15);
  if constexpr (sizeof(T) == 2)
    if (start & 2) return sum_from<T, kInWords>(x, V, mx, table, first, step);
  return start ? sum_from<T, kOnWords>(x, V, mx, table, first, step)
               : sum_from<T, kOnVectors>(x, V, mx, table, first, step);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

// A candidate: its score (ordered(double); 0: none), and what decides between equal
// scores, the larger being better: the lower beam, the larger logit, the lower token (in
// 6, 32 and 24 bits).
constexpr int kTokenBits = 24;
static_assert(kMaxBeams <= 64 && kMaxVocab <= 1 << kTokenBits, "fields of Cand::tie");
struct __align__(16) Cand {
  uint64_t score, tie;
  __device__ __forceinline__ int beam() const { return kMaxBeams - 1 - (int)(tie >> 56); }
  __device__ __forceinline__ int token() const {
    return (1 << kTokenBits) - 1 - (int)(tie & ((1 << kTokenBits) - 1));
  }
  __device__ __forceinline__ float logit() const {
    return unordered((uint32_t)(tie >> kTokenBits));
  }
};
__device__ __forceinline__ uint64_t make_tie(int beam, uint64_t key) {
  return (uint64_t)(kMaxBeams - 1 - beam) << 56 | (key >> 32) << kTokenBits |
         ((uint32_t)key & ((1 << kTokenBits) - 1));
}
__device__ __forceinline__ bool better(const Cand& a, const Cand& b) {
  return (a.score > b.score) | ((a.score == b.score) & (a.tie > b.tie));
}
__device__ __forceinline__ double value(uint64_t o) {
  return __longlong_as_double((long long)(o >> 63 ? o & ~(1ull << 63) : ~o));
}

// One group in shared memory.
struct Group {
  Cand list[kListCap];  // candidates that may be among the K best
  Cand picked[kMaxBeamSelected];
  double sum[kMaxBeams];    // of exp(x - top)
  double off[kMaxBeams];    // -log of it
  double part[kMaxBeams][kWarps];       // sums taken again: this CTA's warps'
  double parts[kMaxJoinCtas][kMaxBeams];  // and, in the first CTA, all CTAs'
  uint64_t held[kListCap];  // the candidates' keys, if there are no more
  float2 table[64];
  float off32[kMaxBeams];   // -logf of it
  float top[kMaxBeams];     // row maximum
  float cum[kMaxBeams];     // beam score; NaN: the beam offers nothing
  uint8_t done[kMaxBeams];  // finished: one candidate, the end token
  uint8_t again[kMaxBeams];
  uint32_t bar[kWarps];
  int count, near, ranked;
};

static_assert(sizeof(Group) <= 47 * 1024, "a group in the default shared memory");

// A candidate's score in 64 bits (0: below fp32's range, none).  The fp32 numbers first, whose
// sum is exact as a rule: where beams have the same sum, logits and beam scores that make
// equal scores make equal numbers.
__device__ __forceinline__ uint64_t score64(const Group& g, int w, float logit) {
  double s = (double)g.cum[w];
  if (!g.done[w]) s = (s + ((double)logit - (double)g.top[w])) + g.off[w];
  return (float)s != -INFINITY ? ordered(s) : 0;
}

// two picks whose beams' sums have to be taken again to tell their order
__device__ __forceinline__ void note_near(Group& g, const Cand& a, const Cand& b) {
  const int x = a.beam(), y = b.beam();
  const double v = value(a.score);
  if (x == y || v - value(b.score) > kNear + 1e-15 * fabs(v)) return;
  g.again[x] = g.again[y] = 1;
  g.near = 1;
}

// barrier of the joining kernel's first eight warps
__device__ __forceinline__ void main_warps_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kBeamThreads) : "memory");
}
// of how many of their threads p holds
__device__ __forceinline__ int main_warps_count(bool p) {
  int n;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %1, 0;\n\tbar.red.popc.u32 %0, 1, %2, q;\n\t}"
      : "=r"(n)
      : "r"((int)p), "n"(kBeamThreads)
      : "memory");
  return n;
}

// The rare ways, out of the way of the usual ones' instructions.
//
// More candidates than there is room for, or than are soon ranked, reach the threshold
// (many equal scores): a piece's candidates are in the scores' order, so the best of all
// pieces' first ones is taken, K times, some 1.7 us each (one group of 4 equal rows of
// 128256 logits: 226 us with K = 128).  A thread has the pieces tid, tid + 256, ...
// and keeps the best of their first ones; `heads` (two words of each piece, those of its
// maximum and sum) counts the taken ones.  Returns the list's length.
__device__ __noinline__ int list_in_order(Group& g, const uint64_t* keys, uint32_t* heads,
                                          int pieces, int S, int end_key, int K) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto first_of = [&](int piece, uint32_t taken, uint64_t key) {
    const int w = piece / S;
    if (isnan(g.cum[w])) return Cand{0, 0};
    if (g.done[w]) {
      if (piece != w * S || taken != 0) return Cand{0, 0};
      key = (uint64_t)(uint32_t)end_key;
    }
    if (key == 0) return Cand{0, 0};
    return Cand{score64(g, w, unordered((uint32_t)(key >> 32))), make_tie(w, key)};
  };
  for (int piece = tid; piece < pieces; piece += kBeamThreads) heads[2 * piece] = 0;
  Cand mine;
  int at;
  auto look = [&] {
    mine = Cand{0, 0};
    at = tid;
#pragma unroll 1
    for (int p0 = tid; p0 < pieces; p0 += kBatch * kBeamThreads) {
      uint32_t taken[kBatch];
      uint64_t key[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int piece = p0 + i * kBeamThreads;
        taken[i] = piece < pieces ? heads[2 * piece] : K;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        key[i] = taken[i] < (uint32_t)K
                     ? __ldcg(keys + (int64_t)(p0 + i * kBeamThreads) * K + taken[i])
                     : 0;
#pragma unroll 1
      for (int i = 0; i < kBatch; ++i) {
        const int piece = p0 + i * kBeamThreads;
        if (piece < pieces) {
          const Cand o = first_of(piece, taken[0], key[0]);
          if (better(o, mine)) {
            mine = o;
            at = piece;
          }
        }
#pragma unroll
        for (int k = 0; k + 1 < kBatch; ++k) {
          taken[k] = taken[k + 1];
          key[k] = key[k + 1];
        }
      }
    }
  };
  look();
  // (the list's last places hold the warps' best, of two rounds in turn)
  static_assert(kMaxBeamSelected + 2 * kWarps <= kListCap, "room for them");
  int n = 0;
#pragma unroll 1
  for (; n < K; ++n) {
    Cand best = mine;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const Cand o{__shfl_xor_sync(~0u, best.score, d), __shfl_xor_sync(~0u, best.tie, d)};
      if (better(o, best)) best = o;
    }
    Cand* room = g.list + kListCap - (n & 1 ? 2 : 1) * kWarps;
    if (lane == 0) room[warp] = best;
    main_warps_sync();
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (better(room[w], best)) best = room[w];
    if (best.score == 0) break;
    if (tid == 0) g.list[n] = best;
    if (mine.score == best.score && mine.tie == best.tie) {
      ++heads[2 * at];
      look();
    }
  }
  main_warps_sync();
  return n;
}
// and, once they are picked, the candidates left out that are close to the last pick
__device__ __noinline__ void note_near_from_all(Group& g, const uint64_t* keys, int n_all,
                                                int per_row, int end_key, const Cand& end) {
  const float end_s = (float)value(end.score);
#pragma unroll 1
  for (int c0 = threadIdx.x; c0 < n_all; c0 += kBatch * kBeamThreads) {
    uint64_t batch[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int c = c0 + i * kBeamThreads;
      batch[i] = c < n_all ? __ldcg(keys + c) : 0;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int c = c0 + i * kBeamThreads, w = c / per_row;
      if (c >= n_all || w == end.beam() || isnan(g.cum[w])) continue;
      if (g.done[w] && c != w * per_row) continue;
      const uint64_t key = g.done[w] ? (uint64_t)(uint32_t)end_key : batch[i];
      if (key == 0) continue;
      const float x = unordered((uint32_t)(key >> 32));
      const float s = g.done[w] ? g.cum[w] : g.cum[w] + ((x - g.top[w]) + g.off32[w]);
      // (in fp32 first: far more than its error and kNear away, as nearly all are)
      if (s < end_s - 1e-4f - 0x1p-18f * (fabsf(s) + fabsf(g.cum[w]) + fabsf(g.off32[w]))) continue;
      const Cand o{score64(g, w, x), make_tie(w, key)};
      if (o.score != 0 && better(end, o)) note_near(g, end, o);
    }
  }
}

// The sums of the rows noted, in two fp32 parts: CTA `rank` of `ranks` takes its share of
// every row, to `parts` of the first CTA.
__device__ __noinline__ void sum_again(Group& g, const BeamArgs& a, int64_t row0, int rank,
                                       int ranks, double* parts) {
  const int tid = threadIdx.x;
  if (tid < 64) {
    const double t = exp2((double)tid / 64);
    g.table[tid] = make_float2((float)t, (float)(t - (double)(float)t));
  }
  main_warps_sync();
  const int first = rank * kBeamThreads + tid, step = ranks * kBeamThreads;
  for (int w = 0; w < a.beam_width; ++w) {
    if (!g.again[w] || g.done[w]) continue;
    const int64_t at = (row0 + w) * a.row_stride;
    double part =
        a.dtype == PA_F32
            ? precise_sum<float>(a.logits, at, a.vocab_size, g.top[w], g.table, first, step)
        : a.dtype == PA_F16
            ? precise_sum<__half>(a.logits, at, a.vocab_size, g.top[w], g.table, first, step)
            : precise_sum<__nv_bfloat16>(a.logits, at, a.vocab_size, g.top[w], g.table, first,
                                         step);
    part = warp_sum(part);
    if ((tid & 31) == 0) g.part[w][tid >> 5] = part;
  }
  main_warps_sync();
  if (tid < a.beam_width && g.again[tid] && !g.done[tid]) {
    double sum = 0.0;
    for (int i = 0; i < kWarps; ++i) sum += g.part[tid][i];
    parts[rank * kMaxBeams + tid] = sum;
  }
}

// One group: the sums of its rows, then the K best of their candidates.
//
// Bound by latency: a chain of short steps, each run once, whose instructions come
// from a cache that the chunk kernel has just filled; so loops are not unrolled, and
// what is rarely needed lies outside.  FP64 units are few: 64-bit scores are computed
// only where they can decide.  An fp32 score and a bound of its error sort out the
// candidates that reach the K-th best score less kNear (some 20 to 50).
//
// A ninth warp takes the logs in 64 bits (a long chain of FP64 operations) while the
// others sort out by fp32 ones.
// Where there are few groups, a cluster of CTAs takes each, all but the first only to
// help with the sums that have to be taken again (64 groups of 4 beams that are copies of
// each other, 128256 bf16 logits: 106 us with four CTAs to a group, 179 with two).
constexpr int kJoinThreads = kBeamThreads + 32;
__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(BeamK p) {
  extern __shared__ __align__(16) char shared[];
  Group& g = *reinterpret_cast<Group*>(shared);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int W = p.a.beam_width, K = p.a.num_selected, S = p.chunks;
  cg::cluster_group team = cg::this_cluster();
  const int rank = (int)team.block_rank(), ranks = (int)team.num_blocks();
  const int64_t group = blockIdx.x / (unsigned)ranks;
  const int64_t row0 = group * W;
  // Barriers of the cluster: 0, all CTAs run; 1, the first one has told the others whether
  // sums have to be taken again, into their memory; 2, they have been.
  if (ranks > 1) team.barrier_arrive();
  if (rank != 0) {
    if (warp == kWarps) return;
    team.barrier_wait();
    team.sync();
    if (g.near) {
      sum_again(g, p.a, row0, rank, ranks, &team.map_shared_rank(&g, 0)->parts[0][0]);
      team.sync();
    }
    return;
  }
  auto tell = [&](bool near) {
    if (ranks == 1) return;
    team.barrier_wait();
    for (int i = tid; i < (ranks - 1) * W; i += kBeamThreads) {
      Group& o = *team.map_shared_rank(&g, 1 + i / W);
      const int w = i % W;
      if (w == 0) o.near = near;
      if (near) {
        o.again[w] = g.again[w];
        o.done[w] = g.done[w];
        o.top[w] = g.top[w];
      }
    }
    team.barrier_arrive();
    if (near) team.barrier_wait();
  };
  if (tid < W) {
    const float cum = p.a.beam_scores[row0 + tid];
    g.cum[tid] = isfinite(cum) ? cum : NAN;
    g.done[tid] = p.a.finished && p.a.finished[row0 + tid];
    g.again[tid] = 0;
  }
  if (tid == 0) g.count = g.near = g.ranked = 0;
  const int per_row = S * K, n_all = W * per_row, n_held = min(n_all, kListCap);
  const uint64_t* keys = p.keys + row0 * per_row;
  const int end_key = ~p.a.end_token;
  // A thread's candidates: the i-th is stride x i modulo an odd number that is prime to
  // the stride, i = tid, tid + 256, ...  Each has some of many pieces and ranks, so that
  // the best ones are in many threads.
  const unsigned modulus = (unsigned)n_all | 1;
  const unsigned c_first = (unsigned)((uint64_t)tid * p.stride % modulus);
  const unsigned c_step = (unsigned)((uint64_t)kBeamThreads * p.stride % modulus);
  __syncthreads();
  pdl_wait();
  // (a finished row's keys are not written, and not used)
  if (warp < kWarps && n_all == n_held)
#pragma unroll 4
    for (int c = tid; c < n_held; c += kBeamThreads) g.held[c] = __ldcg(keys + c);
#pragma unroll 1
  for (int w = warp; w < W; w += kWarps + 1) {
    if (g.done[w]) {
      if (lane == 0) g.sum[w] = 1.0;
      continue;
    }
    const float2* st = p.stats + (row0 + w) * S;
    float m = -INFINITY;
    double sum = 0.0;
    if (S <= 32) {
      const float2 v = lane < S ? __ldcg(st + lane) : make_float2(-INFINITY, 0.f);
      m = v.x;
#pragma unroll
      for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
      if (v.x > -INFINITY) sum = (double)(v.y * expf(v.x - m));
    } else {
#pragma unroll 1
      for (int i = lane; i < S; i += 32) m = fmaxf(m, __ldcg(&st[i].x));
#pragma unroll
      for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
#pragma unroll 1
      for (int i = lane; i < S; i += 32) {
        const float2 v = __ldcg(st + i);
        if (v.x > -INFINITY) sum += (double)(v.y * expf(v.x - m));
      }
    }
    sum = warp_sum(sum);
    if (lane == 0) {
      g.top[w] = m;
      g.sum[w] = sum;
      g.off32[w] = -logf((float)sum);
      if (m == -INFINITY) g.cum[w] = NAN;
    }
  }
  __syncthreads();
  if (warp == kWarps) {
    for (int w = lane; w < W; w += 32) g.off[w] = -log(g.sum[w]);
    asm volatile("bar.arrive 2, %0;" ::"n"(kJoinThreads) : "memory");
    return;
  }
  int got;
#pragma unroll 1
  for (int pass = 0;; ++pass) {
    auto for_mine = [&](auto&& f) {  // f(candidate, its key)
      unsigned c = c_first;
      auto hop = [&] {
        c += c_step;
        if (c >= modulus) c -= modulus;
      };
      if (n_all == n_held) {
#pragma unroll 1
        for (unsigned i = tid; i < modulus; i += kBeamThreads, hop())
          if (c < (unsigned)n_all) f((int)c, g.held[c]);
        return;
      }
#pragma unroll 1
      for (unsigned i = tid; i < modulus; i += kBatch * kBeamThreads) {
        uint64_t batch[kBatch];
        int at[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k, hop()) {
          at[k] = i + k * kBeamThreads < modulus && c < (unsigned)n_all ? (int)c : -1;
          batch[k] = at[k] >= 0 ? __ldcg(keys + at[k]) : 0;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (at[k] >= 0) f(at[k], batch[k]);
      }
    };
    // Every candidate's beam, key, fp32 score and bound of its error, if it is one.
    auto offered = [&](int c, uint64_t held, int* w, uint64_t* key, float* s, float* err) {
      *w = c / per_row;
      const float cum = g.cum[*w];
      if (isnan(cum)) return false;
      if (g.done[*w]) {
        *key = (uint64_t)(uint32_t)end_key;
        *s = cum;
        *err = 0.f;
        return c == *w * per_row;
      }
      *key = held;
      const float d = unordered((uint32_t)(*key >> 32)) - g.top[*w], off = g.off32[*w];
      *s = cum + (d + off);
      // (logf and its argument: 2^-23 of the log, and 2^-24)
      *err = 0x1p-21f * (fabsf(cum) + fabsf(d) + fabsf(off)) + 0x1p-23f;
      return *key != 0;
    };
    // a threshold that K threads' best candidates reach at least, and not many more: the
    // largest score less 1/4, 1/2, 1, ..., then back some of the last step if that was
    // too far (beams' scores may lie far apart, so that no warp stands for the others)
    float mine = -INFINITY;
    for_mine([&](int c, uint64_t held) {
      int w;
      uint64_t key;
      float s, err;
      if (offered(c, held, &w, &key, &s, &err)) mine = fmaxf(mine, s - err);
    });
    const uint32_t wmax = __reduce_max_sync(~0u, ordered(mine));
    if (lane == 0) g.bar[warp] = wmax;
    main_warps_sync();
    const float top = unordered(__reduce_max_sync(~0u, g.bar[lane & (kWarps - 1)]));
    float step = 0.25f, floor_s = top - step;
    int reach = main_warps_count(mine >= floor_s);
#pragma unroll 1
    for (int i = 0; i < 140 && reach < K; ++i) {  // (2^130 is the largest step in fp32)
      step *= 2.f;
      floor_s = top - step;
      reach = main_warps_count(mine >= floor_s);
    }
    float back = step * 0.25f;
#pragma unroll 1
    for (int i = 0; i < 6 && reach > K + K / 2; ++i, back *= 0.5f) {
      const int n = main_warps_count(mine >= floor_s + back);
      if (n < K) continue;
      floor_s += back;
      reach = n;
    }
    floor_s -= 1.25f * (float)kNear + 0x1p-22f * fabsf(floor_s);
    for_mine([&](int c, uint64_t held) {
      int w;
      uint64_t key;
      float s, err;
      if (!offered(c, held, &w, &key, &s, &err) || s + err < floor_s) return;
      const int at = atomicAdd(&g.count, 1);
      if (at < kListCap) g.list[at].tie = make_tie(w, key);
    });
    if (pass == 0)
      asm volatile("bar.sync 2, %0;" ::"n"(kJoinThreads) : "memory");  // (the logs)
    else
      main_warps_sync();
    int n = g.count;
    const bool all_listed = n <= min(kListCap, 4 * K + 128);
    if (all_listed) {
#pragma unroll 1
      for (int i = tid; i < n; i += kBeamThreads)
        g.list[i].score = score64(g, g.list[i].beam(), g.list[i].logit());
      main_warps_sync();
    } else {
      n = list_in_order(g, keys, reinterpret_cast<uint32_t*>(p.stats + row0 * S), W * S, S,
                        end_key, K);
    }
#pragma unroll 1
    for (int i = tid; i < n; i += kBeamThreads) {
      const Cand o = g.list[i];
      if (o.score == 0) continue;
      int rank = 0;
      for (int j = 0; j < n && rank < K; j += 4)
#pragma unroll
        for (int k = 0; k < 4; ++k) rank += j + k < n && better(g.list[j + k], o);
      if (rank < K) {
        g.picked[rank] = o;
        atomicAdd(&g.ranked, 1);
      }
    }
    main_warps_sync();
    got = g.ranked;
    if (pass == 1 || got == 0) break;
    // ---- scores of two beams too close for the fp32 sums: next to each other, or
    // one left out next to the last one picked
    if (tid + 1 < got) note_near(g, g.picked[tid], g.picked[tid + 1]);
    if (got == K) {
      const Cand end = g.picked[K - 1];
      if (!all_listed)
        note_near_from_all(g, keys, n_all, per_row, end_key, end);
      else
#pragma unroll 1
        for (int i = tid; i < n; i += kBeamThreads)
          if (g.list[i].score != 0 && better(end, g.list[i])) note_near(g, end, g.list[i]);
    }
    main_warps_sync();
    if (!g.near) break;
    tell(true);
    sum_again(g, p.a, row0, 0, ranks, &g.parts[0][0]);
    if (ranks > 1)
      team.sync();
    else
      main_warps_sync();
    if (tid < W && g.again[tid] && !g.done[tid]) {
      double sum = 0.0;
      for (int r = 0; r < ranks; ++r) sum += g.parts[r][tid];
      g.off[tid] = -log(sum);
      g.off32[tid] = (float)g.off[tid];
    }
    if (tid == 0) g.count = g.ranked = 0;
    main_warps_sync();
  }
  if (!g.near) tell(false);
  for (int i = tid; i < K; i += kBeamThreads) {
    const int64_t at = group * K + i;
    float score = -INFINITY;
    int parent = -1, token = -1;
    if (i < got) {
      const Cand o = g.picked[i];
      score = (float)value(o.score);
      parent = (int)row0 + o.beam();
      token = o.token();
    }
    p.a.scores[at] = score;
    p.a.parents[at] = parent;
    p.a.tokens[at] = token;
    if (p.a.finished_out) p.a.finished_out[at] = token >= 0 && token == p.a.end_token;
  }
}

template <typename T>
cudaError_t launch_chunks(const BeamK& p, int per_thread, unsigned grid, cudaStream_t stream) {
  constexpr int kN = Pack<T>::kN;
  constexpr int kLongest = sizeof(T) == 4 ? 32 : 64;
  if (per_thread == kLongest)
    beam_chunk_kernel<T, kLongest / kN><<<grid, kBeamThreads, 0, stream>>>(p);
  else if (per_thread == 32)
    beam_chunk_kernel<T, 32 / kN><<<grid, kBeamThreads, 0, stream>>>(p);
  else
    beam_chunk_kernel<T, 8 / kN><<<grid, kBeamThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

namespace {
// chunks of a row by threads of `e` logits
int64_t chunks_of(int vocab_size, int e) {
  return ((int64_t)vocab_size + kBeamAlign - 1 + kBeamThreads * e - 1) / (kBeamThreads * e);
}
int64_t keys_bytes(int64_t pieces, int num_selected) {
  return (pieces * num_selected * 8 + 255) / 256 * 256;
}
constexpr int kFewCtas = 16;  // with fewer, chunks are short
}  // namespace

BeamPlan make_beam_plan(pa_dtype dtype, int num_groups, int beam_width, int vocab_size,
                        int num_selected) {
  BeamPlan b{};
  const int64_t rows = (int64_t)num_groups * beam_width;
  // the longest chunks (32 registers of logits a thread) that make 16 CTAs: fewer pieces are
  // sooner joined, and a CTA's loads are all in flight at once (one group of 4 beams of
  // 128256 bf16 logits 14.5 us in chunks of 2048, 10.0 in chunks of 16384; of 32000 9.4 and
  // 7.7; four groups of 32000 10.0 and 9.0)
  const int longest = dtype == PA_F32 ? 32 : 64;
  b.per_thread = 8;
  for (int e = longest; e > 8 && b.per_thread == 8; e /= 2)
    if (e != 16 && rows * chunks_of(vocab_size, e) >= kFewCtas) b.per_thread = e;
  b.chunks = (int)chunks_of(vocab_size, b.per_thread);
  b.off_stats = keys_bytes(rows * b.chunks, num_selected);
  b.bytes = b.off_stats + rows * b.chunks * 8;
  return b;
}

// Room for any type's plan (fp32 logits are cut into the most chunks) and for that of any
// fewer rows or smaller vocabulary: of the short chunks, four to a long one, there are fewer
// than 4 x 16.
int64_t beam_workspace_bytes(int num_groups, int beam_width, int vocab_size, int num_selected) {
  const int64_t rows = (int64_t)num_groups * beam_width;
  const int64_t few = rows * chunks_of(vocab_size, 8), many = rows * chunks_of(vocab_size, 32);
  const int64_t at_most = few < 4 * (kFewCtas - 1) ? few : 4 * (kFewCtas - 1);
  const int64_t pieces = many > at_most ? many : at_most;
  return keys_bytes(pieces, num_selected) + pieces * 8;
}

cudaError_t launch_beam_select(const BeamArgs& a, const BeamPlan& plan, int num_sms,
                               cudaStream_t stream) {
  const int64_t candidates = (int64_t)a.beam_width * plan.chunks * a.num_selected;
  const unsigned stride = (candidates | 1) % 1000003 ? 1000003u : 1000033u;  // (primes)
  BeamK p{a, plan.chunks, stride, static_cast<uint64_t*>(a.workspace),
          reinterpret_cast<float2*>(static_cast<char*>(a.workspace) + plan.off_stats)};
  const unsigned grid = (unsigned)((int64_t)a.num_groups * a.beam_width * plan.chunks);
  cudaError_t e = a.dtype == PA_F32   ? launch_chunks<float>(p, plan.per_thread, grid, stream)
                  : a.dtype == PA_F16 ? launch_chunks<__half>(p, plan.per_thread, grid, stream)
                                      : launch_chunks<__nv_bfloat16>(p, plan.per_thread, grid,
                                                                     stream);
  if (e != cudaSuccess) return e;
  count_launch();
  // CTAs to a group: one to 16K logits of a row, while all groups' fit the SMs twice (a
  // cluster costs half a microsecond to launch and tell that there is nothing to do)
  unsigned ctas = 1;
  while (ctas < kMaxJoinCtas && (int64_t)a.num_groups * ctas * 2 <= 2 * num_sms &&
         (int64_t)ctas * 2 * 16384 <= a.vocab_size)
    ctas *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.num_groups * ctas);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = sizeof(Group);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ctas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, beam_join_kernel, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace pa
