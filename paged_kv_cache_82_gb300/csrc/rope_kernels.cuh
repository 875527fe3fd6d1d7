// rope_kernels.cuh -- what lies between a layer's QKV projection and its
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
// Bound by HBM: each of q, k, v is read once and written once.  head_dim / 8
// lanes hold one head's row, two groups of 4 elements each: the groups that
// the rotation pairs (i, i + R/2), so that it stays within a lane, and two
// neighbours where nothing turns or neighbours turn.  The row's sum is a few
// shuffles.  8192 tokens of 64 + 8 + 8 heads of 128, bf16 over an E4M3 cache: 59 us,
// 5.5 TB/s (its bytes at the copy rate: 48 us); what is left are the instructions,
// some 15 per element.  64 tokens: 2.2 us.
#pragma once

#include <type_traits>

#include "pa_step.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
// Rows per lane group, and CTAs per SM (64 registers a thread), of a large
// step.  8192 tokens of 64 + 8 + 8 heads of 128, bf16 over an FP8 cache, in us:
// 8 rows 59, 4 rows 66 with four CTAs; 8 rows 63 with three, 16 rows 78; 4 rows 63
// with five.
constexpr int kHeads = 8;
constexpr int kCtas = 4;

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
  uint32_t per_item;             // 2^(32 + shift) / items, rounded up
  int per_item_shift;
};

// A lane's place in a row of kD elements: two groups of four.  pairs = R / 8:
// the first `pairs` lanes hold the groups g and g + pairs that turn together,
// the others neighbours.
struct Place {
  int g[2];
  __device__ __forceinline__ Place(int sub, int pairs) {
    g[0] = sub < pairs ? sub : 2 * sub;
    g[1] = sub < pairs ? sub + pairs : 2 * sub + 1;
  }
  // the lane and the half of it that hold group k
  __device__ __forceinline__ static int lane_of(int k, int pairs) {
    return k < pairs ? k : k < 2 * pairs ? k - pairs : k >> 1;
  }
  __device__ __forceinline__ static int half_of(int k, int pairs) {
    return k < 2 * pairs ? k >= pairs : k & 1;
  }
};

// The lane's 8 elements, as they are read: kVec by 8 or 16 bytes a group.
// Pairs of 16-bit types are taken apart and put together as words.
template <typename T>
struct Row8 {
  static constexpr int kWords = 2 * sizeof(T);
  uint32_t w[kWords];
  template <bool kVec>
  __device__ __forceinline__ void load(const T* row, const Place& at) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const T* src = row + 4 * at.g[k];
      if constexpr (kVec && sizeof(T) == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(src);
        w[2 * k] = u.x;
        w[2 * k + 1] = u.y;
      } else if constexpr (kVec) {
        const uint4 u = *reinterpret_cast<const uint4*>(src);
        w[4 * k] = u.x, w[4 * k + 1] = u.y, w[4 * k + 2] = u.z, w[4 * k + 3] = u.w;
      } else if constexpr (sizeof(T) == 2) {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
        w[2 * k] = h[0] | (uint32_t)h[1] << 16;
        w[2 * k + 1] = h[2] | (uint32_t)h[3] << 16;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * k + i] = reinterpret_cast<const uint32_t*>(src)[i];
      }
    }
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    if constexpr (std::is_same<T, float>::value) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ void round(const float (&x)[8]) {
    if constexpr (std::is_same<T, float>::value) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = pack2<std::is_same<T, __nv_bfloat16>::value>(x[2 * i], x[2 * i + 1]);
    }
  }
  // a row that allows 16-byte stores
  __device__ __forceinline__ void store(T* row, const Place& at) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2*>(row + 4 * at.g[k]) = make_uint2(w[2 * k], w[2 * k + 1]);
      else
        *reinterpret_cast<uint4*>(row + 4 * at.g[k]) =
            make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    }
  }
};

// One lane's 8 elements of token offset o into the page of a cache, by
// pa_reshape_and_cache's rule.  Every lane of the warp calls it; on: this row
// is written.  sub: the lane's number in its row, of lane - sub on.
template <typename T, int kCache, int kD>
__device__ __forceinline__ void cache_row(void* cache, int64_t page, int o, int lane, int sub,
                                          const Place& at, int pairs, const Row8<T>& row,
                                          const Divisor& scale, bool on) {
  if constexpr (kCache == kSame) {
    if (on) row.store(static_cast<T*>(cache) + (page * kBS + o) * kD, at);
    return;
  }
  float x[8], y[8];
  row.values(x);  // of the input type, whatever the cache's
  if constexpr (kCache == kFp8) {
    divide(x, scale, y);
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * k], y[4 * k + 1]),
                                                   __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * k + 2], y[4 * k + 3]),
                                                   __NV_SATFINITE, __NV_E4M3);
      w[k] = lo | hi << 16;
    }
    uint8_t* dst = static_cast<uint8_t*>(cache) + (page * kBS + o) * kD;
    if (on) {
      *reinterpret_cast<uint32_t*>(dst + 4 * at.g[0]) = w[0];
      *reinterpret_cast<uint32_t*>(dst + 4 * at.g[1]) = w[1];
    }
  } else if constexpr (kCache == kInt4) {
    uint8_t* pg = static_cast<uint8_t*>(cache) + page * (8 * kD + 64);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int d = 1; d < kD / 8; d <<= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
    const float sc = amax > 0.f ? __fdiv_rn(amax, 7.0f) : 0.f;
    divide(x, Divisor(sc), y);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int c = sc > 0.f ? __float2int_rn(y[i]) : 0;
      c = max(-7, min(7, c));
      w[i >> 2] |= ((uint32_t)c & 0xFu) << (4 * (i & 3));
    }
    if (on) {
      if (sub == 0) *reinterpret_cast<float*>(pg + kBS * (kD / 2) + 4 * o) = sc;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        *reinterpret_cast<uint16_t*>(pg + o * (kD / 2) + 2 * at.g[k]) = (uint16_t)w[k];
    }
  } else {
    uint8_t* pg = static_cast<uint8_t*>(cache) + page * (9 * kD);
    float own[2] = {0.f, 0.f};  // the groups' largest values
#pragma unroll
    for (int i = 0; i < 8; ++i) own[i >> 2] = fmaxf(own[i >> 2], fabsf(x[i]));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // of the 16-element block: four groups, wherever they are
      const int first = at.g[k] & ~3;
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int from = lane - sub + Place::lane_of(first + j, pairs);
        const float a = __shfl_sync(~0u, own[0], from), b = __shfl_sync(~0u, own[1], from);
        amax = fmaxf(amax, Place::half_of(first + j, pairs) ? b : a);
      }
      const uint8_t bs = static_cast<uint8_t>(__nv_cvt_float_to_fp8(
          __fdiv_rn(__fdiv_rn(amax, 6.0f), scale.s), __NV_SATFINITE, __NV_E4M3));
      const float r = __fmul_rn(e4m3_to_f32(bs), scale.s);
      const float xk[4] = {x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]};
      float yk[4];
      divide(xk, Divisor(r), yk);
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) w |= (r > 0.f ? e2m1_encode(yk[i]) : 0u) << (4 * i);
      if (on) {
        if ((at.g[k] & 3) == 0) pg[kBS * (kD / 2) + o * (kD / 16) + at.g[k] / 4] = bs;
        *reinterpret_cast<uint16_t*>(pg + o * (kD / 2) + 2 * at.g[k]) = (uint16_t)w;
      }
    }
  }
}

// One warp: kH rows per group of lanes, all query, all key or all value heads
// of one token, so the rotation's row and the weights are read once for kH
// heads; all rows are on their way before the first is used.  kVec: rows and
// weights allow 16-byte loads.
template <typename T, int kCache, int kD, bool kInter, bool kVec, int kH>
__global__ void __launch_bounds__(kThreads, kCtas) norm_rope_kernel(const RopeParams p) {
  constexpr int kLanes = kD / 8;      // lanes of one head's row
  constexpr int kRows = 32 / kLanes;  // rows of one warp at a time
  const int lane = threadIdx.x & 31, sub = lane % kLanes;
  const uint32_t warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const uint32_t tok = __umulhi(warp, p.per_item) >> p.per_item_shift;
  const int64_t t = tok;
  if (t >= p.num_tokens) return;
  const int item = (int)(warp - tok * (uint32_t)p.items);
  const int which = item < p.q_items ? 0 : item < p.q_items + p.kv_items ? 1 : 2;
  const int heads = which == 0 ? p.num_q_heads : p.num_kv_heads;
  const int first = (item - (which == 0 ? 0 : p.q_items + (which - 1) * p.kv_items)) *
                    (kRows * kH);
  const int h0 = first + lane / kLanes;
  const int half = p.rotary_dim / 2;
  const int pairs = kInter ? 0 : p.rotary_dim / 8;
  const Place at(sub, pairs);
  // the rows do not depend on the slot: their loads go out together
  const int64_t slot = __ldg(p.slot_mapping + t);
  const int64_t pos = p.rotary_dim ? __ldg(p.positions + t) : 0;
  const T* src = (which == 0   ? static_cast<const T*>(p.q) + t * p.q_stride
                  : which == 1 ? static_cast<const T*>(p.k) + t * p.k_stride
                               : static_cast<const T*>(p.v) + t * p.v_stride) +
                 h0 * kD;
  Row8<T> raw[kH];
#pragma unroll
  for (int j = 0; j < kH; ++j)
    if (h0 + j * kRows < heads) raw[j].template load<kVec>(src + j * kRows * kD, at);
  if (slot < 0) return;  // a padding token: nothing written
  if (slot >= p.num_slots || (p.rotary_dim && (pos < 0 || pos >= p.max_position))) {
    if (item == 0 && lane == 0)
      flag_error(p.err, slot >= p.num_slots ? PA_DEV_ERR_SLOT : PA_DEV_ERR_METADATA);
    return;
  }
  // The lane's rotation with the weights in it: element i of the result is
  //   r (x_i own_i + x_partner other_i),  r = 1/sqrt(mean + eps),
  //   own = w cos, other = -+ w_partner sin
  // (no norm: w = r = 1; no rotation: cos = 1, sin = 0).
  const void* wp = which == 0 ? p.q_weight : which == 1 ? p.k_weight : nullptr;
  const bool turns =
      which < 2 && (kInter ? sub * 8 < p.rotary_dim : sub < pairs);
  float own[8], other[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) own[i] = 1.f, other[i] = 0.f;
  if (turns) {
    const float* row = p.cos_sin + pos * p.rotary_dim + sub * 4;
    const float4 c4 = __ldg(reinterpret_cast<const float4*>(row));
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + half));
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int a = kInter ? 2 * i : i, b = kInter ? 2 * i + 1 : i + 4;
      own[a] = own[b] = c[i];
      other[a] = -s[i];
      other[b] = s[i];
    }
  }
  if (wp) {
    float w[8];
    if (p.weight_f32) {
      Row8<float> r8;
      r8.template load<kVec>(static_cast<const float*>(wp), at);
      r8.values(w);
    } else {
      Row8<T> r8;
      r8.template load<kVec>(static_cast<const T*>(wp), at);
      r8.values(w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      own[i] *= w[i];
      other[i] *= kInter ? w[i ^ 1] : w[i ^ 4];
    }
  }
  const int64_t b = slot / kBS;
  const int o = (int)(slot - b * kBS);
  const Divisor scale(which == 2 ? p.v_scale : p.k_scale,
                      which > 0 && (kCache == kFp8 || kCache == kNvfp4));
  T* q_out = static_cast<T*>(p.q_out) + (t * p.num_q_heads + h0) * kD;
  // Rows of one kind, each straight through: without a branch between them their
  // instructions interleave (the chunk above: 59 us, with branches on the kind and
  // the norm in every row 70).
  auto rows = [&](auto kind, auto norm) {
#pragma unroll
    for (int j = 0; j < kH; ++j) {
      if (first + j * kRows >= heads) break;  // the whole warp is past
      const bool on = h0 + j * kRows < heads;
      if constexpr (kind() < 2) {
        float x[8], y[8];
        raw[j].values(x);
        float r = 1.f;
        if constexpr (norm()) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
          for (int d = 1; d < kLanes; d <<= 1) ss += __shfl_xor_sync(~0u, ss, d);
          r = rsqrtf(ss * (1.0f / kD) + p.eps);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] = x[i] * own[i];
          if (turns) y[i] = fmaf(kInter ? x[i ^ 1] : x[i ^ 4], other[i], y[i]);
          if constexpr (norm()) y[i] *= r;
        }
        raw[j].round(y);
      }
      if constexpr (kind() == 0) {
        if (on) raw[j].store(q_out + j * kRows * kD, at);
      } else {
        cache_row<T, kCache, kD>(kind() == 2 ? p.v_cache : p.k_cache,
                                 b * p.num_kv_heads + h0 + j * kRows, o, lane, sub, at, pairs,
                                 raw[j], scale, on);
      }
    }
  };
  using std::integral_constant;
  if (which == 2)
    rows(integral_constant<int, 2>{}, std::false_type{});
  else if (which == 1 && wp)
    rows(integral_constant<int, 1>{}, std::true_type{});
  else if (which == 1)
    rows(integral_constant<int, 1>{}, std::false_type{});
  else if (wp)
    rows(integral_constant<int, 0>{}, std::true_type{});
  else
    rows(integral_constant<int, 0>{}, std::false_type{});
}

template <typename T, int kCache, int kD, bool kVec, int kH>
cudaError_t launch_h(RopeParams p, cudaStream_t stream) {
  constexpr int kRows = 32 / (kD / 8) * kH;
  p.q_items = (p.num_q_heads + kRows - 1) / kRows;
  p.kv_items = (p.num_kv_heads + kRows - 1) / kRows;
  p.items = p.q_items + 2 * p.kv_items;
  const int64_t blocks =
      (p.num_tokens * p.items + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks >= (1ll << 28)) return cudaErrorInvalidValue;  // warps: 31 bits
  // warp / items by a product (Granlund and Montgomery 1994): with 2^l >= items,
  // l = shift + 1, the factor m = ceil(2^(31 + l) / items) is exact for 31-bit
  // numerators, since m items - 2^(31 + l) < items <= 2^l
  p.per_item_shift = 0;
  while ((2u << p.per_item_shift) < (uint32_t)p.items) ++p.per_item_shift;
  p.per_item = (uint32_t)((((uint64_t)1 << (32 + p.per_item_shift)) + p.items - 1) / p.items);
  if (p.interleaved)
    norm_rope_kernel<T, kCache, kD, true, kVec, kH>
        <<<(unsigned)blocks, kThreads, 0, stream>>>(p);
  else
    norm_rope_kernel<T, kCache, kD, false, kVec, kH>
        <<<(unsigned)blocks, kThreads, 0, stream>>>(p);
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

// The call for inputs of type T (one translation unit each: their many forms
// are compiled side by side).
template <typename T>
cudaError_t launch_rope(const RopeArgs& a, int num_sms, unsigned* err, cudaStream_t stream) {
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
  return launch_c<T>(p, a.cache_dtype, a.head_dim, a.vector_ok, stream);
}

extern template cudaError_t launch_rope<float>(const RopeArgs&, int, unsigned*, cudaStream_t);
extern template cudaError_t launch_rope<__half>(const RopeArgs&, int, unsigned*, cudaStream_t);
extern template cudaError_t launch_rope<__nv_bfloat16>(const RopeArgs&, int, unsigned*,
                                                       cudaStream_t);

}  // namespace pa
