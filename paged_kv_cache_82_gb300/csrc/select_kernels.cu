// select_kernels.cu -- which cache blocks a query reads: per-block bounds of
// the keys (pa_summarise_blocks) and the selection by them (pa_select_blocks).
//
// A block's record holds, per KV head and channel d, the largest and smallest
// key value hi_d, lo_d of its written tokens as 8-bit codes of one scale s
// (rounded outwards).  For a query q, sum_d max(q_d hi_d, q_d lo_d) is then at
// least the score of the block's best key: the block's own bound, for 1/32 of
// the bytes of its bf16 K and V pages.
//
// The query is quantised to 8 bits too (one scale for the query heads of a KV
// head), so a bound is a sum of whole numbers below 2^24 and the score
// fl32(s * max over the heads of the sum) has one rounding: it does not depend
// on the order of the sum, and equal inputs select equal blocks everywhere.
#include <float.h>
#include <limits.h>

#include <algorithm>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;

constexpr int bounds_bytes(int d) { return PA_BOUNDS_BYTES(d); }

// ---------------------------------------------------------------------------
// pa_summarise_blocks
// ---------------------------------------------------------------------------
enum : int { kPgF32 = 0, kPgF16, kPgBf16, kPgFp8, kPgInt4, kPgNvfp4 };

// 8 consecutive channels (from 8 * c8) of the token at offset o of a page
template <int kPg, int kD>
__device__ __forceinline__ void page_load8(const void* cache, int64_t page, int o,
                                           int c8, float (&x)[8]) {
  if constexpr (kPg == kPgF32) {
    const float4* src = reinterpret_cast<const float4*>(
        static_cast<const float*>(cache) + (page * kBS + o) * kD + c8 * 8);
    const float4 a = __ldg(src), b = __ldg(src + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else if constexpr (kPg == kPgF16 || kPg == kPgBf16) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(
        static_cast<const uint16_t*>(cache) + (page * kBS + o) * kD + c8 * 8));
    if constexpr (kPg == kPgF16) {
      const __half* e = reinterpret_cast<const __half*>(&u);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = to_f32(e[i]);
    } else {
      const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(&u);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = to_f32(e[i]);
    }
  } else if constexpr (kPg == kPgFp8) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(
        static_cast<const uint8_t*>(cache) + (page * kBS + o) * kD + c8 * 8));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = e4m3_to_f32((uint8_t)((i < 4 ? u.x : u.y) >> (8 * (i & 3))));
  } else {
    constexpr int kPage = kPg == kPgNvfp4 ? 9 * kD : 8 * kD + 64;
    const uint8_t* pg = static_cast<const uint8_t*>(cache) + page * kPage;
    const uint32_t w =
        __ldg(reinterpret_cast<const uint32_t*>(pg + o * (kD / 2) + c8 * 4));
    if constexpr (kPg == kPgInt4) {
      const float sc = __ldg(reinterpret_cast<const float*>(pg + kBS * (kD / 2) + 4 * o));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = sc * (float)((int)(w << (28 - 4 * i)) >> 28);
    } else {
      const float sc =
          e4m3_to_f32(__ldg(pg + kBS * (kD / 2) + o * (kD / 16) + c8 / 2));
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = sc * e2m1_to_f32((w >> (4 * i)) & 15u);
    }
  }
}

// One group of kD / 8 lanes per (written block, KV head): 8 channels per lane,
// the block's tokens one after the other.
template <int kPg, int kD>
__global__ void __launch_bounds__(kThreads)
summarise_kernel(StepView s, const void* __restrict__ k_cache, int num_kv_heads,
                 int groups_per_seq, uint8_t* __restrict__ bounds) {
  constexpr int kLanes = kD / 8, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, sub = lane % kLanes;
  const int64_t warp = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int64_t item = warp * kRows + lane / kLanes;
  const int64_t per_seq = (int64_t)groups_per_seq * num_kv_heads;
  if (item >= per_seq * s.num_seqs) return;
  const int r = (int)(item / per_seq);
  const int rem = (int)(item - r * per_seq);
  const int nth = rem / num_kv_heads, h = rem - nth * num_kv_heads;
  const ReqMeta m = load_req(s.query_start_loc, s.seq_lens, r, s.num_tokens,
                             s.max_query_len, s.max_seq_len, s.max_blocks_per_seq);
  if (!m.ok) {
    if (rem == 0 && sub == 0) flag_error(s.err, PA_DEV_ERR_METADATA);
    return;
  }
  const int b = (m.L - m.n) / kBS + nth;  // the nth block this step wrote to
  if (m.n == 0 || b >= m.nb) return;
  const int blk = __ldg(s.block_tables + (int64_t)r * s.max_blocks_per_seq + b);
  if (blk < 0 || (int64_t)blk >= s.num_blocks) {
    if (h == 0 && sub == 0) flag_error(s.err, PA_DEV_ERR_BLOCK_ID);
    return;
  }
  const int64_t page = (int64_t)blk * num_kv_heads + h;
  const int tokens = min(kBS, m.L - b * kBS);
  float hi[8], lo[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) hi[i] = -INFINITY, lo[i] = INFINITY;
#pragma unroll 4
  for (int o = 0; o < tokens; ++o) {
    float x[8];
    page_load8<kPg, kD>(k_cache, page, o, sub, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // a NaN is passed over
      hi[i] = fmaxf(hi[i], x[i]);
      lo[i] = fminf(lo[i], x[i]);
    }
  }
  float big = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (lo[i] > hi[i]) lo[i] = hi[i] = 0.f;  // nothing but NaN in the channel
    lo[i] = fminf(fmaxf(lo[i], -FLT_MAX), FLT_MAX);
    hi[i] = fminf(fmaxf(hi[i], -FLT_MAX), FLT_MAX);
    big = fmaxf(big, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
  }
  const unsigned mask = kLanes == 32 ? ~0u : ((1u << kLanes) - 1) << (lane - sub);
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) big = fmaxf(big, __shfl_xor_sync(mask, big, d));
  const float sc = __fdiv_rn(big, 127.0f);
  uint32_t ch[2] = {0, 0}, cl[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int a = sc > 0.f ? min(127, max(-127, __float2int_ru(__fdiv_rn(hi[i], sc)))) : 0;
    const int c = sc > 0.f ? min(127, max(-127, __float2int_rd(__fdiv_rn(lo[i], sc)))) : 0;
    ch[i >> 2] |= ((uint32_t)a & 0xFFu) << (8 * (i & 3));
    cl[i >> 2] |= ((uint32_t)c & 0xFFu) << (8 * (i & 3));
  }
  uint8_t* rec = bounds + page * bounds_bytes(kD);
  *reinterpret_cast<uint2*>(rec + sub * 8) = make_uint2(ch[0], ch[1]);
  *reinterpret_cast<uint2*>(rec + kD + sub * 8) = make_uint2(cl[0], cl[1]);
  if (sub == 0)
    *reinterpret_cast<uint4*>(rec + 2 * kD) = make_uint4(__float_as_uint(sc), 0, 0, 0);
}

// ---------------------------------------------------------------------------
// pa_select_blocks: scores
// ---------------------------------------------------------------------------
// fp32 order as unsigned order
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr uint32_t kKeptKey = 0xFFFFFFFFu;  // above every score's key

struct ScoreParams {
  StepView s;
  int64_t t0;  // first token of the pass
  const void* q;
  int num_q_heads, num_kv_heads, group;
  const uint8_t* bounds;
  int max_selected, keep_first, keep_last;
  int64_t row_scores;
  uint32_t* keys;  // [token of the pass][KV head][row_scores]
};

// Token t's request, position and visible blocks; -1 blocks: none (a token of
// no request, or broken metadata, which is flagged if tell).
struct TokenView {
  int r, pos, blocks;
};
__device__ __forceinline__ TokenView token_view(const StepView& s, int64_t t, bool tell) {
  TokenView v{0, 0, -1};
  v.r = warp_find_request(s.query_start_loc, s.num_seqs, t);
  const ReqMeta m = load_req(s.query_start_loc, s.seq_lens, v.r, s.num_tokens,
                             s.max_query_len, s.max_seq_len, s.max_blocks_per_seq);
  if (t < m.q0 || t >= (int64_t)m.q0 + m.n) return v;
  if (!m.ok) {
    if (tell) flag_error(s.err, PA_DEV_ERR_METADATA);
    return v;
  }
  v.pos = m.L - m.n + (int)(t - m.q0);
  v.blocks = v.pos / kBS + 1;
  return v;
}

constexpr int kScoreWarps = 8;
constexpr int kScoreBlocks = 64;  // cache blocks of one CTA

// One CTA: one token, kScoreBlocks cache blocks, all KV heads (a warp per
// head in turn: the heads' records of a block are one contiguous range).
// kD / 16 lanes hold a record's 16 channels each, so a warp reads 512 / kD
// records at a time; the query's codes stay in registers.
template <typename TQ, int kD, int kG>
__global__ void __launch_bounds__(kScoreWarps * 32) score_kernel(const ScoreParams p) {
  constexpr int kLanes = kD / 16;
  constexpr int kRecs = 32 / kLanes;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % kLanes;
  const int64_t t = p.t0 + blockIdx.y;
  const int first = (int)blockIdx.x * kScoreBlocks;
  const TokenView tv = token_view(p.s, t, false);
  if (tv.blocks <= p.max_selected || first >= tv.blocks) return;  // all of them
  const int last = min(first + kScoreBlocks, tv.blocks);
  const int32_t* table = p.s.block_tables + (int64_t)tv.r * p.s.max_blocks_per_seq;
  for (int h = warp; h < p.num_kv_heads; h += kScoreWarps) {
    const TQ* qp = static_cast<const TQ*>(p.q) +
                   (t * p.num_q_heads + (int64_t)h * p.group) * kD + sub * 16;
    // one scale for all heads of the group
    float big = 0.f;
    for (int g = 0; g < p.group; ++g)
#pragma unroll
      for (int i = 0; i < 16; ++i) big = fmaxf(big, fabsf(to_f32(qp[g * kD + i])));
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, d));
    const float sq = __fdiv_rn(big, 127.0f);
    uint32_t* keys = p.keys + ((int64_t)blockIdx.y * p.num_kv_heads + h) * p.row_scores;
    for (int b0 = first; b0 < last; b0 += kRecs) {
      const int b = b0 + lane / kLanes;
      const bool kept = b < p.keep_first || b >= tv.blocks - p.keep_last;
      int blk = b < last && !kept ? __ldg(table + b) : 0;
      if (blk < 0 || (int64_t)blk >= p.s.num_blocks) {
        if (sub == 0 && h == 0) flag_error(p.s.err, PA_DEV_ERR_BLOCK_ID);
        blk = 0;
      }
      const uint8_t* rec = p.bounds + ((int64_t)blk * p.num_kv_heads + h) * bounds_bytes(kD);
      const uint4 hi = __ldg(reinterpret_cast<const uint4*>(rec + sub * 16));
      const uint4 lo = __ldg(reinterpret_cast<const uint4*>(rec + kD + sub * 16));
      const float sc = __ldg(reinterpret_cast<const float*>(rec + 2 * kD));
      const uint32_t hw[4] = {hi.x, hi.y, hi.z, hi.w}, lw[4] = {lo.x, lo.y, lo.z, lo.w};
      int best = INT_MIN;
      for (int g = 0; g < p.group; ++g) {
        int dot = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t code = 0, neg = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = to_f32(qp[g * kD + 4 * w + i]);
            int c = sq > 0.f ? __float2int_rn(__fdiv_rn(x, sq)) : 0;
            c = min(127, max(-127, c));
            code |= ((uint32_t)c & 0xFFu) << (8 * i);
            neg |= (c < 0 ? 0xFFu : 0u) << (8 * i);
          }
          dot = __dp4a((int)((hw[w] & ~neg) | (lw[w] & neg)), (int)code, dot);
        }
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) dot += __shfl_xor_sync(~0u, dot, d);
        best = max(best, dot);
      }
      // + 0: a zero is a positive zero
      if (sub == 0 && b < last)
        keys[b] = kept ? kKeptKey : order_key(__fmul_rn((float)best, sc) + 0.0f);
    }
  }
}

// ---------------------------------------------------------------------------
// pa_select_blocks: the K largest keys, ties to the lowest block
// ---------------------------------------------------------------------------
struct TopkParams {
  StepView s;
  int64_t t0;
  int num_kv_heads, max_selected;
  int64_t row_scores;
  const uint32_t* keys;
  int32_t* selected;
  int32_t* num_selected;
};

constexpr int kTopkThreads = 256;

__global__ void __launch_bounds__(kTopkThreads) topk_kernel(const TopkParams p) {
  __shared__ int hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  __shared__ int warp_above[kTopkThreads / 32], warp_equal[kTopkThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = (int)(blockIdx.x % p.num_kv_heads);
  const int64_t tp = blockIdx.x / p.num_kv_heads, t = p.t0 + tp;
  const TokenView tv = token_view(p.s, t, h == 0 && tid == 0);
  if (tv.blocks < 0) return;
  const int64_t row = t * p.num_kv_heads + h;
  int32_t* out = p.selected + row * p.max_selected;
  const int K = p.max_selected, n = tv.blocks;
  if (tid == 0) p.num_selected[row] = min(n, K);
  if (n <= K) {
    for (int i = tid; i < K; i += kTopkThreads) out[i] = i < n ? i : -1;
    return;
  }
  const uint32_t* keys = p.keys + (tp * p.num_kv_heads + h) * p.row_scores;
  // the K-th largest key, 8 bits at a time from the top
  uint32_t prefix = 0;
  int need = K;
  for (int shift = 24; shift >= 0; shift -= 8) {
    hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kTopkThreads) {
      const uint32_t k = keys[i];
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l owns bins 8 l .. 8 l + 7; keys in the lanes above it
      int own = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) own += hist[lane * 8 + i];
      int above = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_down_sync(~0u, above, d);
        if (lane + d < 32) above += o;
      }
      above -= own;
      if (above < need && above + own >= need) {
        for (int i = 7; i >= 0; --i) {
          const int c = hist[lane * 8 + i];
          if (above + c >= need) {
            s_prefix = prefix | (uint32_t)(lane * 8 + i) << shift;
            s_need = need - above;
            break;
          }
          above += c;
        }
      }
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // in order: the keys above, and the first `need` of the equal ones.  Each
  // warp has a contiguous part of the row.
  constexpr int kWarps = kTopkThreads / 32;
  const int part = ((n + kWarps - 1) / kWarps + 31) & ~31;
  const int lo = min(n, warp * part), hi = min(n, lo + part);
  int above = 0, equal = 0;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < hi ? keys[i] : 0u;
    above += __popc(__ballot_sync(~0u, i < hi && k > prefix));
    equal += __popc(__ballot_sync(~0u, i < hi && k == prefix));
  }
  if (lane == 0) warp_above[warp] = above, warp_equal[warp] = equal;
  __syncthreads();
  int at = 0, eq = 0;  // entries before this warp's part
  for (int w = 0; w < warp; ++w) {
    at += warp_above[w];
    eq += warp_equal[w];
  }
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < hi ? keys[i] : 0u;
    const unsigned gt = __ballot_sync(~0u, i < hi && k > prefix);
    const unsigned ge = __ballot_sync(~0u, i < hi && k == prefix);
    const unsigned below = (1u << lane) - 1;
    const int e = eq + __popc(ge & below);  // equal keys before this one
    if ((gt >> lane & 1) || ((ge >> lane & 1) && e < need))
      out[at + __popc(gt & below) + min(e, need)] = i;
    at += __popc(gt);
    eq += __popc(ge);
  }
}

template <int kPg, int kD>
cudaError_t launch_summarise_d(const StepView& s, const void* k_cache, int num_kv_heads,
                               void* bounds, cudaStream_t stream) {
  // blocks a request of max_query_len tokens writes to, at most
  const int64_t wide = std::min<int64_t>((s.max_query_len + kBS - 2) / kBS + 1,
                                         (s.max_seq_len + kBS - 1) / kBS);
  const int64_t items = wide * num_kv_heads * s.num_seqs;
  const int64_t per_block = kThreads / (kD / 8);
  const int64_t blocks = (items + per_block - 1) / per_block;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  summarise_kernel<kPg, kD><<<(unsigned)blocks, kThreads, 0, stream>>>(
      s, k_cache, num_kv_heads, (int)wide, static_cast<uint8_t*>(bounds));
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

template <int kPg>
cudaError_t launch_summarise_t(const StepView& s, const void* k_cache, int num_kv_heads,
                               int head_dim, void* bounds, cudaStream_t stream) {
  return head_dim == 128
             ? launch_summarise_d<kPg, 128>(s, k_cache, num_kv_heads, bounds, stream)
             : launch_summarise_d<kPg, 64>(s, k_cache, num_kv_heads, bounds, stream);
}

template <typename TQ>
cudaError_t launch_score(const ScoreParams& p, int head_dim, dim3 grid,
                         cudaStream_t stream) {
  if (head_dim == 128)
    score_kernel<TQ, 128, 1><<<grid, kScoreWarps * 32, 0, stream>>>(p);
  else
    score_kernel<TQ, 64, 1><<<grid, kScoreWarps * 32, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

cudaError_t launch_summarise_blocks(const StepView& s, const void* k_cache,
                                    pa_dtype cache_dtype, int num_kv_heads,
                                    int head_dim, void* bounds, cudaStream_t stream) {
  switch (cache_dtype) {
    case PA_F32:
      return launch_summarise_t<kPgF32>(s, k_cache, num_kv_heads, head_dim, bounds, stream);
    case PA_F16:
      return launch_summarise_t<kPgF16>(s, k_cache, num_kv_heads, head_dim, bounds, stream);
    case PA_BF16:
      return launch_summarise_t<kPgBf16>(s, k_cache, num_kv_heads, head_dim, bounds, stream);
    case PA_FP8_E4M3:
      return launch_summarise_t<kPgFp8>(s, k_cache, num_kv_heads, head_dim, bounds, stream);
    case PA_INT4:
      return launch_summarise_t<kPgInt4>(s, k_cache, num_kv_heads, head_dim, bounds, stream);
    case PA_NVFP4:
      return launch_summarise_t<kPgNvfp4>(s, k_cache, num_kv_heads, head_dim, bounds,
                                          stream);
  }
  return cudaErrorInvalidValue;
}

SelectPlan make_select_plan(int64_t num_tokens, int num_kv_heads, int max_seq_len) {
  SelectPlan pl{};
  const int64_t blocks = ((int64_t)max_seq_len + kBS - 1) / kBS;
  pl.row_scores = (blocks + 3) / 4 * 4;
  const int64_t token_bytes = pl.row_scores * num_kv_heads * 4;
  pl.pass_tokens = token_bytes > 0 ? kSelectScoreBytes / token_bytes : num_tokens;
  pl.pass_tokens = std::max<int64_t>(1, std::min<int64_t>(pl.pass_tokens, 32768));
  pl.pass_tokens = std::min(pl.pass_tokens, num_tokens);
  pl.bytes = pl.pass_tokens * token_bytes;
  return pl;
}

cudaError_t launch_select_blocks(const StepView& s, const SelectPlan& plan,
                                 const void* q, pa_dtype q_dtype, int num_q_heads,
                                 int num_kv_heads, int head_dim, const void* bounds,
                                 int max_selected, int keep_first, int keep_last,
                                 int32_t* selected, int32_t* num_selected,
                                 void* workspace, int num_sms, cudaStream_t stream) {
  const int max_blocks = (s.max_seq_len + kBS - 1) / kBS;
  for (int64_t t0 = 0; t0 < s.num_tokens; t0 += plan.pass_tokens) {
    const int64_t nt = std::min(plan.pass_tokens, s.num_tokens - t0);
    if (max_blocks > max_selected) {
      ScoreParams p{};
      p.s = s;
      p.t0 = t0;
      p.q = q;
      p.num_q_heads = num_q_heads;
      p.num_kv_heads = num_kv_heads;
      p.group = num_q_heads / num_kv_heads;
      p.bounds = static_cast<const uint8_t*>(bounds);
      p.max_selected = max_selected;
      p.keep_first = keep_first;
      p.keep_last = keep_last;
      p.row_scores = plan.row_scores;
      p.keys = static_cast<uint32_t*>(workspace);
      const dim3 grid((unsigned)((max_blocks + kScoreBlocks - 1) / kScoreBlocks),
                      (unsigned)nt);
      cudaError_t e;
      switch (q_dtype) {
        case PA_F32: e = launch_score<float>(p, head_dim, grid, stream); break;
        case PA_F16: e = launch_score<__half>(p, head_dim, grid, stream); break;
        default: e = launch_score<__nv_bfloat16>(p, head_dim, grid, stream); break;
      }
      if (e != cudaSuccess) return e;
    }
    TopkParams tp{};
    tp.s = s;
    tp.t0 = t0;
    tp.num_kv_heads = num_kv_heads;
    tp.max_selected = max_selected;
    tp.row_scores = plan.row_scores;
    tp.keys = static_cast<const uint32_t*>(workspace);
    tp.selected = selected;
    tp.num_selected = num_selected;
    if (nt * num_kv_heads > 0x7fffffffll) return cudaErrorInvalidValue;
    topk_kernel<<<(unsigned)(nt * num_kv_heads), kTopkThreads, 0, stream>>>(tp);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launch();
  }
  return cudaSuccess;
}

}  // namespace pa
