// rope_kernels.cu -- what lies between a layer's QKV projection and its
// attention, in one pass (pa_norm_rope_and_cache): RMS norm of every query and
// key head, the position rotation, and the write of K and V into the cache.
//
//   y = x * 1/sqrt(mean(x^2) + eps) * w                       (with weights)
//   (a, b) -> (a cos - b sin, b cos + a sin) over the first rotary_dim
//   dimensions, pairs (i, i + R/2) or, interleaved, (2i, 2i + 1)
//
// all in fp32, rounded once to the input type; a key then goes through
// pa_reshape_and_cache's rule for the cache type, so that the result is the
// two-step result bit for bit.
//
// Bound by HBM: each of q, k, v is read once and written once.  A group of
// head_dim / 8 lanes holds one head's row, 8 elements (16 bytes of a 16-bit
// type) per lane: the row's sum is a few shuffles, and the rotation's partner
// of element i lies in the lane rotary_dim / 16 away at the same place (or,
// interleaved, in the same lane).
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
#ifndef PA_ROPE_CTAS
#define PA_ROPE_CTAS 4
#endif
#ifndef PA_ROPE_H
#define PA_ROPE_H 4
#endif
constexpr int kHeads = PA_ROPE_H;  // rows per lane group of a large step

enum : int { kSame = 0, kFp8 = 1, kInt4 = 2, kNvfp4 = 3 };

struct RopeParams {
  const void* q;
  const void* k;
  const void* v;
  int64_t num_tokens, q_stride, k_stride, v_stride;
  const void* q_weight;
  const void* k_weight;
  int weight_f32;
  float eps;
  const float* cos_sin;
  int64_t max_position;
  int rotary_dim, interleaved;
  const int32_t* positions;
  void* q_out;
  void* k_cache;
  void* v_cache;
  int64_t num_slots;
  int num_q_heads, num_kv_heads;
  const int64_t* slot_mapping;
  float k_scale, v_scale;
  unsigned* err;
  int num_sms;
  int items, q_items, kv_items;  // warps of one token: all, per kind
};

// 8 consecutive elements as fp32
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* src, float (&x)[8]) {
  if constexpr (kVec && sizeof(T) == 2) {
    const uint4 u = *reinterpret_cast<const uint4*>(src);
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(e[i]);
  } else if constexpr (kVec) {
    const float4 a = *reinterpret_cast<const float4*>(src);
    const float4 b = *reinterpret_cast<const float4*>(src + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(src[i]);
  }
}

// 8 consecutive elements (16-byte aligned), rounded to T
template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint4 u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(x[i]);
    *reinterpret_cast<uint4*>(dst) = u;
  } else {
    *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// 8 elements of a row as they are read, 16 or 32 bytes
template <typename T>
struct alignas(16) Row8 {
  T e[8];
  template <bool kVec>
  __device__ __forceinline__ void load(const T* src) {
    if constexpr (kVec) {
      const uint4* s = reinterpret_cast<const uint4*>(src);
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(e)[i] = s[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = src[i];
    }
  }
  __device__ __forceinline__ Row8 shuffled(int from) const {
    Row8 o;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) * 2; ++i)
      reinterpret_cast<uint32_t*>(o.e)[i] =
          __shfl_sync(~0u, reinterpret_cast<const uint32_t*>(e)[i], from);
    return o;
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(e[i]);
  }
};

// One lane's 8 elements x (lane sub of the kD / 8 of a row) of token offset o
// into the page of a cache, by pa_reshape_and_cache's rule.  Every lane of
// the warp calls it; on: this row is written.
template <typename T, int kCache, int kD>
__device__ __forceinline__ void cache_row(void* cache, int64_t page, int o, int sub,
                                          float (&x)[8], const Divisor& scale, bool on) {
  if constexpr (kCache == kSame) {
    if (on) store8(static_cast<T*>(cache) + (page * kBS + o) * kD + sub * 8, x);
  } else if constexpr (kCache == kFp8) {
    float y[8];
    divide(x, scale, y);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c = __nv_cvt_float_to_fp8(y[i], __NV_SATFINITE, __NV_E4M3);
      w[i >> 2] |= c << (8 * (i & 3));
    }
    if (on)
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + (page * kBS + o) * kD +
                                sub * 8) = make_uint2(w[0], w[1]);
  } else {
    constexpr int kPage = kCache == kNvfp4 ? 9 * kD : 8 * kD + 64;
    // a row's (INT4) or a 16-element block's (NVFP4: two lanes) largest value
    constexpr int kLanes = kCache == kNvfp4 ? 2 : kD / 8;
    float amax = 0.f, y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
    uint8_t* pg = static_cast<uint8_t*>(cache) + page * kPage;
    uint32_t codes = 0;
    if constexpr (kCache == kInt4) {
      const float sc = amax > 0.f ? __fdiv_rn(amax, 7.0f) : 0.f;
      divide(x, Divisor(sc), y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        int c = sc > 0.f ? __float2int_rn(y[i]) : 0;
        c = max(-7, min(7, c));
        codes |= ((uint32_t)c & 0xFu) << (4 * i);
      }
      if (on && sub == 0) *reinterpret_cast<float*>(pg + kBS * (kD / 2) + 4 * o) = sc;
    } else {
      const uint8_t bs = static_cast<uint8_t>(__nv_cvt_float_to_fp8(
          __fdiv_rn(__fdiv_rn(amax, 6.0f), scale.s), __NV_SATFINITE, __NV_E4M3));
      const float r = __fmul_rn(e4m3_to_f32(bs), scale.s);
      divide(x, Divisor(r), y);
#pragma unroll
      for (int i = 0; i < 8; ++i) codes |= (r > 0.f ? e2m1_encode(y[i]) : 0u) << (4 * i);
      if (on && (sub & 1) == 0) pg[kBS * (kD / 2) + o * (kD / 16) + sub / 2] = bs;
    }
    // element 2i in the low nibble of byte i: nibble i of the word
    if (on) *reinterpret_cast<uint32_t*>(pg + o * (kD / 2) + sub * 4) = codes;
  }
}

// One warp: kH rows per group of lanes, all query, all key or all value heads
// of one token, so the rotation's row and the weights are read once for kH
// heads; all rows are on their way before the first is used.  kVec: rows and
// weights allow 16-byte loads.
template <typename T, int kCache, int kD, bool kVec, int kH>
__global__ void __launch_bounds__(kThreads, PA_ROPE_CTAS) norm_rope_kernel(const RopeParams p) {
  constexpr int kLanes = kD / 8;      // lanes of one head's row
  constexpr int kRows = 32 / kLanes;  // rows of one warp at a time
  const int lane = threadIdx.x & 31, sub = lane % kLanes;
  const uint32_t warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = warp / (uint32_t)p.items;
  if (t >= p.num_tokens) return;
  const int item = (int)(warp - (uint32_t)t * (uint32_t)p.items);
  const int which = item < p.q_items ? 0 : item < p.q_items + p.kv_items ? 1 : 2;
  const int heads = which == 0 ? p.num_q_heads : p.num_kv_heads;
  const int h0 = (item - (which == 0 ? 0 : p.q_items + (which - 1) * p.kv_items)) *
                     (kRows * kH) + lane / kLanes;
  const int64_t slot = __ldg(p.slot_mapping + t);
  const int64_t pos = p.rotary_dim ? __ldg(p.positions + t) : 0;
  const T* src = (which == 0   ? static_cast<const T*>(p.q) + t * p.q_stride
                  : which == 1 ? static_cast<const T*>(p.k) + t * p.k_stride
                               : static_cast<const T*>(p.v) + t * p.v_stride) +
                 sub * 8;
  // the rows do not depend on the slot: their loads go out together
  Row8<T> raw[kH];
#pragma unroll
  for (int j = 0; j < kH; ++j) {
    const int h = h0 + j * kRows;
    if (h < heads) raw[j].template load<kVec>(src + (int64_t)h * kD);
  }
  if (slot < 0) return;  // a padding token: nothing written
  if (slot >= p.num_slots || (p.rotary_dim && (pos < 0 || pos >= p.max_position))) {
    if (item == 0 && lane == 0)
      flag_error(p.err, slot >= p.num_slots ? PA_DEV_ERR_SLOT : PA_DEV_ERR_METADATA);
    return;
  }
  // The lane's rotation with the weights in it: element i of the result is
  //   r (x_i own_i + x_partner other_i),  r = 1/sqrt(mean + eps),
  //   own = w cos, other = -+ w_partner sin
  // (no norm: w = r = 1; no rotation: cos = 1, sin = 0).  The partner's element
  // comes as it was read: a shuffle of the packed row.
  const void* wp = which == 0 ? p.q_weight : which == 1 ? p.k_weight : nullptr;
  const int half = p.rotary_dim / 2;
  const bool turns = which < 2 && sub * 8 < p.rotary_dim;
  const bool second = sub * 8 >= half;
  const int away = p.rotary_dim / 16;  // lanes between the two of a pair
  const int partner = !turns || p.interleaved ? sub : second ? sub - away : sub + away;
  float own[8], other[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) own[i] = 1.f, other[i] = 0.f;
  if (turns) {
    const float* row = p.cos_sin + pos * p.rotary_dim;
    if (p.interleaved) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + sub * 4));
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + sub * 4));
      own[0] = own[1] = c.x, own[2] = own[3] = c.y;
      own[4] = own[5] = c.z, own[6] = own[7] = c.w;
      other[0] = -s.x, other[1] = s.x, other[2] = -s.y, other[3] = s.y;
      other[4] = -s.z, other[5] = s.z, other[6] = -s.w, other[7] = s.w;
    } else {
      const int f = sub * 8 - (second ? half : 0);
      const float4* cp = reinterpret_cast<const float4*>(row + f);
      const float4* sp = reinterpret_cast<const float4*>(row + half + f);
      *reinterpret_cast<float4*>(own) = __ldg(cp);
      *reinterpret_cast<float4*>(own + 4) = __ldg(cp + 1);
      *reinterpret_cast<float4*>(other) = __ldg(sp);
      *reinterpret_cast<float4*>(other + 4) = __ldg(sp + 1);
      if (!second)
#pragma unroll
        for (int i = 0; i < 8; ++i) other[i] = -other[i];
    }
  }
  if (wp) {
    float w[8], v[8];
    if (p.weight_f32) {
      load8<float, kVec>(static_cast<const float*>(wp) + sub * 8, w);
      load8<float, kVec>(static_cast<const float*>(wp) + partner * 8, v);
    } else {
      load8<T, kVec>(static_cast<const T*>(wp) + sub * 8, w);
      load8<T, kVec>(static_cast<const T*>(wp) + partner * 8, v);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      own[i] *= w[i];
      other[i] *= p.interleaved ? w[i ^ 1] : v[i];
    }
  }
  const int from = (lane - sub) + partner;
  const int64_t b = slot / kBS;
  const int o = (int)(slot - b * kBS);
  const Divisor scale(which == 2 ? p.v_scale : p.k_scale);
#pragma unroll
  for (int j = 0; j < kH; ++j) {
    if (h0 - lane / kLanes + j * kRows >= heads) break;  // the whole warp is past
    const int h = h0 + j * kRows;
    const bool on = h < heads;
    float x[8];
    raw[j].values(x);
    float r = 1.f;
    if (wp) {
      float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 v = make_float2(x[i], x[i + 1]);
        s2 = fma2(v, v, s2);
      }
      float ss = s2.x + s2.y;
#pragma unroll
      for (int d = 1; d < kLanes; d <<= 1) ss += __shfl_xor_sync(~0u, ss, d);
      r = rsqrtf(ss * (1.0f / kD) + p.eps);
    }
    if (which < 2) {
      float y[8];
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
      } else if (p.rotary_dim) {
        raw[j].shuffled(from).values(y);
      }
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        float2 z = mul2(make_float2(x[i], x[i + 1]), make_float2(own[i], own[i + 1]));
        if (turns)
          z = fma2(make_float2(y[i], y[i + 1]), make_float2(other[i], other[i + 1]), z);
        z = mul2(z, make_float2(r, r));
        x[i] = z.x;
        x[i + 1] = z.y;
      }
    }
    if (which == 0) {
      if (on) store8(static_cast<T*>(p.q_out) + (t * p.num_q_heads + h) * kD + sub * 8, x);
    } else {
      // the stored key is that of the input type, whatever the cache's
      if constexpr (kCache != kSame) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = to_f32(from_f32<T>(x[i]));
      }
      cache_row<T, kCache, kD>(which == 2 ? p.v_cache : p.k_cache,
                               b * p.num_kv_heads + h, o, sub, x,
                               scale, on);
    }
  }
}

template <typename T, int kCache, int kD, bool kVec, int kH>
cudaError_t launch_h(RopeParams p, cudaStream_t stream) {
  constexpr int kRows = 32 / (kD / 8) * kH;
  p.q_items = (p.num_q_heads + kRows - 1) / kRows;
  p.kv_items = (p.num_kv_heads + kRows - 1) / kRows;
  p.items = p.q_items + 2 * p.kv_items;
  const int64_t blocks =
      (p.num_tokens * p.items + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks >= (1ll << 29)) return cudaErrorInvalidValue;  // warps: 32 bits
  norm_rope_kernel<T, kCache, kD, kVec, kH><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename T, int kCache, int kD>
cudaError_t launch_d(const RopeParams& p, bool vec, cudaStream_t stream) {
  if (!vec) return launch_h<T, kCache, kD, false, 1>(p, stream);
  // several heads per lane group once that still leaves every SM 16 warps
  const int64_t rows = p.num_tokens * (p.num_q_heads + 2 * p.num_kv_heads);
  if (rows >= 16ll * p.num_sms * kHeads * (32 / (kD / 8)))
    return launch_h<T, kCache, kD, true, kHeads>(p, stream);
  return launch_h<T, kCache, kD, true, 1>(p, stream);
}

template <typename T, int kCache>
cudaError_t launch_t(const RopeParams& p, int head_dim, bool vec, cudaStream_t stream) {
  return head_dim == 128 ? launch_d<T, kCache, 128>(p, vec, stream)
                         : launch_d<T, kCache, 64>(p, vec, stream);
}

template <typename T>
cudaError_t launch_c(const RopeParams& p, pa_dtype cache, int head_dim, bool vec,
                     cudaStream_t stream) {
  switch (cache) {
    case PA_FP8_E4M3: return launch_t<T, kFp8>(p, head_dim, vec, stream);
    case PA_INT4: return launch_t<T, kInt4>(p, head_dim, vec, stream);
    case PA_NVFP4: return launch_t<T, kNvfp4>(p, head_dim, vec, stream);
    default: return launch_t<T, kSame>(p, head_dim, vec, stream);
  }
}

}  // namespace

cudaError_t launch_norm_rope_and_cache(const RopeArgs& a, int num_sms, unsigned* err,
                                       cudaStream_t stream) {
  RopeParams p{};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.num_tokens = a.num_tokens;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.q_weight = a.q_weight;
  p.k_weight = a.k_weight;
  p.weight_f32 = a.weight_dtype == PA_F32;
  p.eps = a.eps;
  p.cos_sin = a.cos_sin;
  p.max_position = a.max_position;
  p.rotary_dim = a.rotary_dim;
  p.interleaved = a.interleaved;
  p.positions = a.positions;
  p.q_out = a.q_out;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.num_slots = a.num_blocks * kBS;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.slot_mapping = a.slot_mapping;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.err = err;
  p.num_sms = num_sms;
  switch (a.dtype) {
    case PA_F32: return launch_c<float>(p, a.cache_dtype, a.head_dim, a.vector_ok, stream);
    case PA_F16: return launch_c<__half>(p, a.cache_dtype, a.head_dim, a.vector_ok, stream);
    case PA_BF16:
      return launch_c<__nv_bfloat16>(p, a.cache_dtype, a.head_dim, a.vector_ok, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
