// select_kernels.cu -- which cache blocks a query reads: per-block bounds of
// the keys (pa_summarise_blocks) and the selection by them (pa_select_blocks).
//
// A block's record holds, per KV head and channel d, the largest and smallest
// key value hi_d, lo_d of its written tokens as 8-bit codes of one scale s
// (rounded outwards).  For a query q, sum_d max(q_d hi_d, q_d lo_d) is then at
// least the score of the block's best key: the block's own bound, for 1/30 of
// the bytes of its bf16 K and V pages.
//
// The query is quantised to 8 bits too (one scale for the query heads of a KV
// head), so a bound is a sum of whole numbers below 2^24 and the score
// fl32(s * max over the heads of the sum) has one rounding: it does not depend
// on the order of the sum, and equal inputs select equal blocks everywhere.
#include <float.h>
#include <limits.h>

#include <algorithm>

#include "pa_step.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;

constexpr int bounds_bytes(int d) { return PA_BOUNDS_BYTES(d); }

// ---------------------------------------------------------------------------
// pa_summarise_blocks
// ---------------------------------------------------------------------------
enum : int { kPgF32 = 0, kPgF16, kPgBf16, kPgFp8, kPgInt4, kPgNvfp4 };

// A lane's 8 consecutive channels of one token of a page, as read
template <int kPg>
struct PageWords {
  static constexpr int kWords = kPg == kPgF32                        ? 8
                                : kPg == kPgF16 || kPg == kPgBf16 ? 4
                                : kPg == kPgFp8                      ? 2
                                                                     : 1;
  uint32_t w[kWords];
  float scale;  // 4-bit pages: the token's or the block's
};

template <int kPg, int kD>
__device__ __forceinline__ PageWords<kPg> page_words(const void* cache, int64_t page, int o,
                                                     int c8) {
  PageWords<kPg> v;
  v.scale = 0.f;
  if constexpr (kPg == kPgF32) {
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const float*>(cache) + (page * kBS + o) * kD + c8 * 8);
    *reinterpret_cast<uint4*>(v.w) = __ldg(src);
    *reinterpret_cast<uint4*>(v.w + 4) = __ldg(src + 1);
  } else if constexpr (kPg == kPgF16 || kPg == kPgBf16) {
    *reinterpret_cast<uint4*>(v.w) = __ldg(reinterpret_cast<const uint4*>(
        static_cast<const uint16_t*>(cache) + (page * kBS + o) * kD + c8 * 8));
  } else if constexpr (kPg == kPgFp8) {
    *reinterpret_cast<uint2*>(v.w) = __ldg(reinterpret_cast<const uint2*>(
        static_cast<const uint8_t*>(cache) + (page * kBS + o) * kD + c8 * 8));
  } else {
    constexpr int kPage = kPg == kPgNvfp4 ? 9 * kD : 8 * kD + 64;
    const uint8_t* pg = static_cast<const uint8_t*>(cache) + page * kPage;
    v.w[0] = __ldg(reinterpret_cast<const uint32_t*>(pg + o * (kD / 2) + c8 * 4));
    if constexpr (kPg == kPgInt4)
      v.scale = __ldg(reinterpret_cast<const float*>(pg + kBS * (kD / 2) + 4 * o));
    else
      v.scale = e4m3_to_f32(__ldg(pg + kBS * (kD / 2) + o * (kD / 16) + c8 / 2));
  }
  return v;
}

// Running largest and smallest of 8 channels: packed pairs where the page's
// values are 16-bit numbers (E4M3 as f16), fp32 elsewhere.  A NaN is passed
// over, as fmaxf and the packed maximum do.
template <int kPg>
struct Range8 {
  static constexpr bool kPair = kPg == kPgF16 || kPg == kPgBf16 || kPg == kPgFp8;
  static constexpr bool kBF = kPg == kPgBf16;
  static constexpr int kN = kPair ? 4 : 8;
  uint32_t hi[kN], lo[kN];

  __device__ __forceinline__ static uint32_t max_of(uint32_t a, uint32_t b) {
    if constexpr (!kPair) {
      return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    } else if constexpr (kBF) {
      const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                       *reinterpret_cast<__nv_bfloat162*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    } else {
      const __half2 m =
          __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    }
  }
  __device__ __forceinline__ static uint32_t min_of(uint32_t a, uint32_t b) {
    if constexpr (!kPair) {
      return __float_as_uint(fminf(__uint_as_float(a), __uint_as_float(b)));
    } else if constexpr (kBF) {
      const __nv_bfloat162 m = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                       *reinterpret_cast<__nv_bfloat162*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    } else {
      const __half2 m =
          __hmin2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    }
  }
  __device__ __forceinline__ void clear() {
    const uint32_t inf = !kPair ? 0x7F800000u : kBF ? 0x7F807F80u : 0x7C007C00u;
    const uint32_t ninf = !kPair ? 0xFF800000u : kBF ? 0xFF80FF80u : 0xFC00FC00u;
#pragma unroll
    for (int i = 0; i < kN; ++i) hi[i] = ninf, lo[i] = inf;
  }
  __device__ __forceinline__ void add(const PageWords<kPg>& v) {
    uint32_t x[kN];
    if constexpr (kPg == kPgFp8) {
      e4m3x4_to_f16x2x2(v.w[0], x[0], x[1]);
      e4m3x4_to_f16x2x2(v.w[1], x[2], x[3]);
    } else if constexpr (kPair || kPg == kPgF32) {
#pragma unroll
      for (int i = 0; i < kN; ++i) x[i] = v.w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t nib = (v.w[0] >> (4 * i)) & 15u;
        x[i] = __float_as_uint(v.scale * (kPg == kPgInt4 ? (float)((int)(nib ^ 8u) - 8)
                                                         : e2m1_to_f32(nib)));
      }
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      hi[i] = max_of(hi[i], x[i]);
      lo[i] = min_of(lo[i], x[i]);
    }
  }
  // with the lane `mask` away
  __device__ __forceinline__ void join(int mask) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      hi[i] = max_of(hi[i], __shfl_xor_sync(~0u, hi[i], mask));
      lo[i] = min_of(lo[i], __shfl_xor_sync(~0u, lo[i], mask));
    }
  }
  __device__ __forceinline__ static uint32_t abs_of(uint32_t a) {
    if constexpr (!kPair) {
      return a & 0x7FFFFFFFu;
    } else if constexpr (kBF) {
      const __nv_bfloat162 m = __habs2(*reinterpret_cast<__nv_bfloat162*>(&a));
      return *reinterpret_cast<const uint32_t*>(&m);
    } else {
      const __half2 m = __habs2(*reinterpret_cast<__half2*>(&a));
      return *reinterpret_cast<const uint32_t*>(&m);
    }
  }
  // the largest magnitude among the lane's channels
  __device__ __forceinline__ float largest() const {
    uint32_t m = max_of(abs_of(hi[0]), abs_of(lo[0]));
#pragma unroll
    for (int i = 1; i < kN; ++i) m = max_of(m, max_of(abs_of(hi[i]), abs_of(lo[i])));
    if constexpr (!kPair) return __uint_as_float(m);
    const uint32_t w[kN] = {m};
    return fmaxf(value(w, 0), value(w, 1));
  }
  __device__ __forceinline__ static float value(const uint32_t (&w)[kN], int i) {
    if constexpr (!kPair) {
      return __uint_as_float(w[i]);
    } else if constexpr (kBF) {
      return __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    } else {
      const __half2 h = *reinterpret_cast<const __half2*>(&w[i / 2]);
      return (i & 1) ? __high2float(h) : __low2float(h);
    }
  }
};

// One warp per (written block, KV head): kD / 8 lanes hold 8 channels each of
// a token, the warp reads 256 / kD tokens at a time and all of the page's 16
// before it uses the first.  The page is read once and a 1/32 to 1/8 of its
// bytes written, so the kernel is bound by HBM when there are many pages, and
// by the chain of loads (lengths, block id, page) when there are few.  16 x 32K
// tokens x 8 heads of 128, E4M3: 109 us, 5.6 TB/s; one block of 64 requests: 2.6 us.
template <int kPg, int kD>
__device__ __forceinline__ void summarise_one(const StepView& s, const void* k_cache,
                                              int num_kv_heads, int r, int nth, int h,
                                              uint8_t* bounds) {
  constexpr int kLanes = kD / 8, kRows = 32 / kLanes, kReads = kBS / kRows;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, part = lane / kLanes;
  const ReqMeta m = load_req(s.query_start_loc, s.seq_lens, r, s.num_tokens,
                             s.max_query_len, s.max_seq_len, s.max_blocks_per_seq);
  if (!m.ok) {
    if (nth == 0 && h == 0 && lane == 0) flag_error(s.err, PA_DEV_ERR_METADATA);
    return;
  }
  const int b = (m.L - m.n) / kBS + nth;  // the nth block this step wrote to
  if (m.n == 0 || b >= m.nb) return;
  const int blk = __ldg(s.block_tables + (int64_t)r * s.max_blocks_per_seq + b);
  if (blk < 0 || (int64_t)blk >= s.num_blocks) {
    if (h == 0 && lane == 0) flag_error(s.err, PA_DEV_ERR_BLOCK_ID);
    return;
  }
  const int64_t page = (int64_t)blk * num_kv_heads + h;
  const int tokens = min(kBS, m.L - b * kBS);
  // a place past the block's tokens reads its last token again
  PageWords<kPg> words[kReads];
  if (tokens == kBS) {
#pragma unroll
    for (int i = 0; i < kReads; ++i)
      words[i] = page_words<kPg, kD>(k_cache, page, i * kRows + part, sub);
  } else {
#pragma unroll
    for (int i = 0; i < kReads; ++i)
      words[i] = page_words<kPg, kD>(k_cache, page, min(i * kRows + part, tokens - 1), sub);
  }
  using Range = Range8<kPg>;
  Range range;
  range.clear();
#pragma unroll
  for (int i = 0; i < kReads; ++i) range.add(words[i]);
#pragma unroll
  for (int d = kLanes; d < 32; d <<= 1) range.join(d);
  float big = range.largest();
  // The first part of the warp has the codes of the largest values, the second
  // those of the smallest: ceil(hi / s) and -ceil(lo / -s).
  const bool low = part & 1;
  float x[8];
  {
    uint32_t w[Range::kN];
#pragma unroll
    for (int i = 0; i < Range::kN; ++i) w[i] = low ? range.lo[i] : range.hi[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = Range::value(w, i);
  }
  // infinite: an infinite key, or a channel of nothing but NaN (hi -inf, lo inf)
  if (big == INFINITY) {
    big = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float hi = Range::value(range.hi, i), lo = Range::value(range.lo, i);
      x[i] = lo > hi ? 0.f : fminf(fmaxf(x[i], -FLT_MAX), FLT_MAX);
      if (lo <= hi)
        big = fmaxf(big, fminf(fmaxf(fabsf(lo), fabsf(hi)), FLT_MAX));
    }
  }
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, d));
  const float sc = __fdiv_rn(big, 127.0f);
  // fp32 keys may be as small as 2^-149: their quotients are divided out
  const Divisor by(sc, kPg != kPgF32);
  const float s1 = low ? -sc : sc, rcp = low ? -by.rcp : by.rcp;
  // c = 1.5 x 2^23 + ceil(q) by a sum rounded up: the code is its lowest byte.
  // The smallest values' sign turns about 1.5 x 2^23.
  constexpr float kUnit = 12582912.0f;
  const float turn = low ? -1.f : 1.f, about = low ? 2 * kUnit : 0.f;
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float q;
    if (by.easy) {
      // Divisor's two corrections; |x| <= 127.01 s, so nothing overflows, and a
      // zero's sign does not matter
      q = x[i] * rcp;
      q = fmaf(fmaf(-q, s1, x[i]), rcp, q);
      q = fmaf(fmaf(-q, s1, x[i]), rcp, q);
    } else {
      // (a scale that is a subnormal of few bits may leave a quotient well past 127,
      // of either sign)
      q = sc > 0.f ? fmaxf(__fdiv_rn(x[i], s1), -127.0f) : 0.f;
    }
    c[i] = __float_as_uint(fmaf(__fadd_ru(fminf(q, 127.0f), kUnit), turn, about));
  }
  uint32_t code[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    code[k] = __byte_perm(__byte_perm(c[4 * k], c[4 * k + 1], 0x0040),
                          __byte_perm(c[4 * k + 2], c[4 * k + 3], 0x0040), 0x5410);
  uint8_t* rec = bounds + page * bounds_bytes(kD);
  if (part < 2)
    *reinterpret_cast<uint2*>(rec + (low ? kD : 0) + sub * 8) = make_uint2(code[0], code[1]);
  if (lane == 0)
    *reinterpret_cast<uint4*>(rec + 2 * kD) = make_uint4(__float_as_uint(sc), 0, 0, 0);
}

template <int kPg, int kD>
__global__ void __launch_bounds__(kThreads)
summarise_kernel(StepView s, const void* __restrict__ k_cache, int num_kv_heads,
                 uint8_t* __restrict__ bounds) {
  const int nth = blockIdx.x, h = blockIdx.z * (blockDim.x / 32) + (threadIdx.x >> 5);
  if (h >= num_kv_heads) return;
  for (int r = blockIdx.y; r < s.num_seqs; r += gridDim.y)
    summarise_one<kPg, kD>(s, k_cache, num_kv_heads, r, nth, h, bounds);
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
// a score's key; a NaN's (of a record that was never written) is the highest
// (named: the sign of a NaN's bits may be changed as a number's, which keeps none)
__device__ __forceinline__ uint32_t score_key(float x) {
  return isnan(x) ? kKeptKey - 1 : order_key(x);
}

struct ScoreParams {
  StepView s;
  int64_t t0;  // first token of the pass
  const void* q;
  int num_q_heads, num_kv_heads, group;
  const uint8_t* bounds;
  int max_selected, keep_first, keep_last;
  int chunk;  // cache blocks of one CTA
  int64_t row_scores;
  uint32_t* keys;  // [token of the pass][KV head][row_scores]
};

// Token t's request, position and visible blocks; -1 blocks: none (a token of
// no request, or broken metadata, which check_requests flags).
struct TokenView {
  int r, pos, blocks;
};
__device__ __forceinline__ TokenView token_view(const StepView& s, int64_t t) {
  TokenView v{0, 0, -1};
  const TokenReq q =
      warp_token_request(s.query_start_loc, s.seq_lens, s.num_seqs, t, s.num_tokens,
                         s.max_query_len, s.max_seq_len, s.max_blocks_per_seq);
  if (!q.in || !q.m.ok) return v;
  v.r = q.r;
  v.pos = q.m.L - q.m.n + (int)(t - q.m.q0);
  v.blocks = v.pos / kBS + 1;
  return v;
}

// each byte's sign bit all over the byte
__device__ __forceinline__ uint32_t sign_bytes(uint32_t x) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %1, 0xba98;" : "=r"(d) : "r"(x));
  return d;
}

// d += a b: 16 rows (records) x 32 codes, times 32 codes x 8 columns (heads), in
// whole numbers
__device__ __forceinline__ void mma_codes(int (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// four 8 x 8 matrices of 16-bit pairs: their rows' addresses in lanes 0-7, 8-15, ..
__device__ __forceinline__ void load_matrices(uint32_t (&a)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(at)
               : "memory");
}

// 4 consecutive elements as fp32 (aligned to as much)
template <typename T>
__device__ __forceinline__ void load4(const T* src, float* x) {
  if constexpr (sizeof(T) == 4) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(src));
    x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
  } else {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(src));
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = to_f32(e[j]);
  }
}

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

constexpr int kScoreWarps = 8;
constexpr int kScoreGroup = 16;  // records a warp stages and scores at a time
// Buffers of a warp, and CTAs per SM: 64 rows of 8 heads x 512 to 4096 blocks,
// both kernels, 59 us with 2 and 3, 68 with 3 and 2 or with 2 and 2.
constexpr int kScoreBufs = 2;
constexpr int kScoreCtas = 3;
// Blocks of one CTA with a warp to each head; as many times more where several
// warps share one: 59 us with 128, 60 with 256, 62 with 64 (each warp codes its
// query anew); one KV head, 29 us with 256, 34 with 128.  Where that leaves fewer
// than four CTAs per SM, down to kScoreChunkMin: one row of 8192 blocks 13.9 us
// with 32, 15.1 with 16 or 64.
constexpr int kScoreChunkMax = 128, kScoreChunkMin = 32;
constexpr int kScoreHeads = 8;   // query heads scored at a time

template <int kD>
struct ScoreLayout {
  static constexpr int kRec = PA_BOUNDS_BYTES(kD);
  static constexpr int kBuf = kScoreGroup * kRec;  // bytes
  static constexpr int kWarp = kScoreBufs * kBuf;
  static constexpr int kSmem = kScoreWarps * kWarp;
};

// One CTA: one token, p.chunk cache blocks, up to eight KV heads.  A warp takes
// one head (the heads' records of a block are one contiguous range, read by the
// CTA's warps at about the same time); with fewer heads than warps, several
// warps share a head's blocks.
//
// Each warp copies 16 records at a time into shared memory of its own, the
// next ones while it scores these, so that what is on its way does not wait
// for registers.  The sum over the channels of a code times the bound of its
// side is a product of 2 kD columns: the records' hi codes times the positive
// codes of the query, and their lo codes times the negative ones (0 elsewhere).
// 16 records by 8 query heads by 32 codes are one integer MMA, whose operands a
// record's row and the codes in a lane's registers are; a record's 17 (or 9)
// words of 16 bytes put eight rows into different banks.  GB300's integer MMAs are
// slow beside its others, and still quicker than the same sums by dp4a with the
// bound picked by the code's sign: 64 tokens of 8K to 64K, both kernels, 8 query
// heads per KV head 63 us (dp4a 83), 5 heads 41 (51), 12 heads 34 (41), 4 heads 59
// (60).
//
// The last one's 232 MB take 48 us of it: 6.3 TB/s while it streams, after 4 to 5
// us for the first records and codes, and before a ragged end.  Neither a third
// buffer nor equal shares of all rows' blocks on resident CTAs (each token's start
// then costs as much) made it shorter.
//
// kFew: up to four query heads, which are columns 0-3 and once more 4-7; the two
// lanes of a head's channels then code half of them each.
template <typename TQ, int kD, bool kFew>
__global__ void __launch_bounds__(kScoreWarps * 32, kScoreCtas)
score_kernel(const ScoreParams p) {
  using Ly = ScoreLayout<kD>;
  constexpr int kSteps = kD / 32;                     // MMAs of a side
  constexpr int kCoded = kFew ? kSteps : 2 * kSteps;  // words of codes a lane makes
  constexpr int kCodePieces = kD / 8;             // 16-byte pieces of a record's codes
  constexpr int kCodeRecs = 32 / kCodePieces;
  extern __shared__ __align__(16) uint8_t score_smem[];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = p.t0 + blockIdx.y;
  const int first = (int)blockIdx.x * p.chunk;
  const int head0 = blockIdx.z * kScoreWarps;
  const int num_heads = min(kScoreWarps, p.num_kv_heads - head0);  // of the CTA
  const int sharing = kScoreWarps / num_heads;                     // warps of one head
  const TokenView tv = token_view(p.s, t);
  if (tv.blocks <= p.max_selected || first >= tv.blocks) return;  // all of them
  if (warp >= sharing * num_heads) return;
  const int h = head0 + warp % num_heads;
  const int last = min(first + p.chunk, tv.blocks);
  const int kept_last = tv.blocks - p.keep_last;
  const int32_t* table = p.s.block_tables + (int64_t)tv.r * p.s.max_blocks_per_seq;
  uint8_t* bufs = score_smem + warp * Ly::kWarp;
  const uint32_t bufs_at = smem_u32(bufs);
  // this lane's record, and its row of the four matrices of an operand
  const int mine = lane & 15;
  const uint32_t row_at = mine * Ly::kRec + (lane >> 4) * 16;
  const int code_off = lane % kCodePieces * 16;
  const uint32_t code_at = lane / kCodePieces * Ly::kRec + code_off;
  const int passes = (p.group + kScoreHeads - 1) / kScoreHeads;
  const int stride = sharing * kScoreGroup;
  const int b_first = first + (warp / num_heads) * kScoreGroup;
  const uint8_t* head_bounds = p.bounds + (int64_t)h * Ly::kRec;
  const int64_t block_bytes = (int64_t)p.num_kv_heads * Ly::kRec;
  // the physical block of block b; -1: kept (not read), none, or out of range
  auto block_id = [&](int b) {
    if (b >= last || b < p.keep_first || b >= kept_last) return -1;
    const int id = __ldg(table + b);
    if (id >= 0 && (int64_t)id < p.s.num_blocks) return id;
    flag_error(p.s.err, PA_DEV_ERR_BLOCK_ID);
    return -1;
  };
  // Copies of the 16 records from block b on: kCodeRecs records' codes at a
  // time, then their scales.  A block that is not read has block 0's.
  auto stage = [&](int b, int buf) {
    int id = -1;
    if (b >= last) {
      copy_commit();
      return id;
    }
    id = block_id(b + mine);
    const int from = max(id, 0);
    const uint32_t dst = bufs_at + buf * Ly::kBuf;
#pragma unroll
    for (int k = 0; k < kScoreGroup; k += kCodeRecs)
      copy16_async(dst + code_at + k * Ly::kRec,
                   head_bounds + code_off +
                       __shfl_sync(~0u, from, k + lane / kCodePieces) * block_bytes);
    if (lane < kScoreGroup)
      copy16_async(dst + lane * Ly::kRec + 2 * kD, head_bounds + 2 * kD + from * block_bytes);
    copy_commit();
    return id;
  };
  int ids[kScoreBufs];
#pragma unroll
  for (int k = 0; k < kScoreBufs - 1; ++k) ids[k] = stage(b_first + k * stride, k);

  const TQ* qp = static_cast<const TQ*>(p.q) +
                 (t * p.num_q_heads + (int64_t)h * p.group) * kD;
  // this lane's head of a pass (past the group's end: its last head again), and
  // its channels: 4 from 32 j + 4 column and from 16 further on
  const int column = lane & 3, head = kFew ? lane >> 2 & 3 : lane >> 2;
  const int coded = kFew ? lane / 16 * kCoded : 0;  // the first of the words
  auto load_query = [&](int pass, float (&x)[4 * kCoded]) {
    const TQ* src = qp + (int64_t)min(pass * kScoreHeads + head, p.group - 1) * kD +
                    4 * column + 16 * coded;
#pragma unroll
    for (int i = 0; i < kCoded; ++i) load4(src + 16 * i, x + 4 * i);
  };
  // one scale for all heads of the group
  float x[4 * kCoded], big = 0.f;
  for (int pass = passes - 1; pass >= 0; --pass) {
    load_query(pass, x);
#pragma unroll
    for (int i = 0; i < 4 * kCoded; ++i) big = fmaxf(big, fabsf(x[i]));
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, d));
  const float sq = __fdiv_rn(big, 127.0f);
  const Divisor by(sq);
  uint32_t* keys = p.keys + ((int64_t)blockIdx.y * p.num_kv_heads + h) * p.row_scores;
  for (int pass = 0; pass < passes; ++pass) {
    if (pass > 0) {
#pragma unroll
      for (int k = 0; k < kScoreBufs - 1; ++k) ids[k] = stage(b_first + k * stride, k);
    }
    // the codes of the lane's head: positive ones, negative ones
    uint32_t up[2 * kSteps], down[2 * kSteps];
    if (pass > 0) load_query(pass, x);
#pragma unroll
    for (int w = 0; w < kCoded; ++w) {
      const float x4[4] = {x[4 * w], x[4 * w + 1], x[4 * w + 2], x[4 * w + 3]};
      float y[4];
      divide(x4, by, y);
      uint32_t c4 = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int c = sq > 0.f ? __float2int_rn(y[i]) : 0;
        c = min(127, max(-127, c));
        c4 |= ((uint32_t)c & 0xFFu) << (8 * i);
      }
      up[w] = c4;
    }
    if constexpr (kFew) {
#pragma unroll
      for (int w = 0; w < kCoded; ++w) {
        const uint32_t other = __shfl_xor_sync(~0u, up[w], 16);
        up[w + kCoded] = coded ? up[w] : other;
        up[w] = coded ? other : up[w];
      }
    }
#pragma unroll
    for (int w = 0; w < 2 * kSteps; ++w) {
      const uint32_t neg = sign_bytes(up[w]);
      down[w] = up[w] & neg;
      up[w] &= ~neg;
    }
    int buf = 0;
    for (int b0 = b_first; b0 < last; b0 += stride) {
      const int id = ids[0];
#pragma unroll
      for (int k = 0; k + 1 < kScoreBufs; ++k) ids[k] = ids[k + 1];
      {
        const int to = buf + kScoreBufs - 1;
        ids[kScoreBufs - 2] = stage(b0 + (kScoreBufs - 1) * stride,
                                    to >= kScoreBufs ? to - kScoreBufs : to);
      }
      copy_wait<kScoreBufs - 1>();
      __syncwarp();
      const uint32_t rows = bufs_at + buf * Ly::kBuf + row_at;
      int hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        uint32_t a[4];
        load_matrices(a, rows + 32 * j);
        mma_codes(hi, a, up[2 * j], up[2 * j + 1]);
        load_matrices(a, rows + kD + 32 * j);
        mma_codes(lo, a, down[2 * j], down[2 * j + 1]);
      }
      const float sc =
          *reinterpret_cast<const float*>(bufs + buf * Ly::kBuf + mine * Ly::kRec + 2 * kD);
      __syncwarp();  // the buffer may be copied into again
      // rows lane / 4 and that + 8, heads 2 column and that + 1
      int top = max(hi[0] + lo[0], hi[1] + lo[1]), low = max(hi[2] + lo[2], hi[3] + lo[3]);
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        top = max(top, __shfl_xor_sync(~0u, top, d));
        low = max(low, __shfl_xor_sync(~0u, low, d));
      }
      top = __shfl_sync(~0u, top, (lane & 7) * 4);
      low = __shfl_sync(~0u, low, (lane & 7) * 4);
      int best = lane & 8 ? low : top;
      const int b = b0 + mine;
      if (lane < kScoreGroup && b < last) {
        uint32_t key;
        if (b < p.keep_first || b >= kept_last) {
          key = kKeptKey;
        } else if (id < 0) {
          key = score_key(-INFINITY);
        } else {
          if (pass > 0) best = max(best, (int)keys[b]);
          // + 0: a zero is a positive zero
          key = pass + 1 < passes ? (uint32_t)best
                                  : score_key(__fmul_rn((float)best, sc) + 0.0f);
        }
        keys[b] = key;
      }
      buf = buf + 1 == kScoreBufs ? 0 : buf + 1;
    }
    copy_wait<0>();
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// pa_select_blocks: the K largest keys, ties to the lowest block
// ---------------------------------------------------------------------------
struct TopkParams {
  StepView s;
  int64_t t0;
  int num_kv_heads, max_selected, kept;  // kept: keep_first + keep_last
  int64_t row_scores;
  const uint32_t* keys;
  int32_t* selected;
  int32_t* num_selected;
};

constexpr int kTopkBits = 10;  // of a key per round
constexpr int kTopkBins = 1 << kTopkBits;

// One CTA per (token, KV head).  The keys' range is cut into 1024 bins, the
// bin that the K-th largest falls into becomes the next range, until a round
// leaves only keys that are all taken (two or three rounds: the first range
// is that of the row's own keys, so no round is spent on their common bits).
// Then each warp writes the entries of its contiguous part of the row in
// order.  kPer keys per lane are held in registers (kTopkThreads x kPer blocks);
// kPer = 0 reads them again each time.  Bound by the rounds' barriers: 512 rows of
// 512 to 4096 blocks about 10 us, 8 rows of 8192 about 7.
template <int kTopkThreads, int kPer>
__global__ void __launch_bounds__(kTopkThreads, 65536 / kTopkThreads / (kPer > 16 ? 80 : 64))
topk_kernel(const TopkParams p) {
  constexpr int kTopkWarps = kTopkThreads / 32;
  constexpr int kTopkOwn = kTopkBins / kTopkThreads;  // bins of a thread
  __shared__ int hist[kTopkBins];
  __shared__ uint32_t s_lo[kTopkWarps], s_hi[kTopkWarps];
  __shared__ int s_warp[kTopkWarps], s_equal[kTopkWarps];
  __shared__ int s_bin, s_need, s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = (int)(blockIdx.x % p.num_kv_heads);
  const int64_t tp = blockIdx.x / p.num_kv_heads, t = p.t0 + tp;
  const TokenView tv = token_view(p.s, t);
  if (p.t0 == 0)
    check_requests(p.s, (int64_t)blockIdx.x * kTopkThreads + tid,
                   (int64_t)gridDim.x * kTopkThreads);
  pdl_wait();  // the scores
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
  // the warp's part: part keys from begin on, 32 at a time
  const int part = ((n + kTopkWarps - 1) / kTopkWarps + 31) & ~31;
  const int begin = min(n, warp * part), end = min(n, begin + part);
  uint32_t held[kPer ? kPer : 1];
  if constexpr (kPer > 0) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = begin + 32 * j + lane;
      held[j] = i < end ? keys[i] : kKeptKey;
    }
  }
  // f(key, block) for each of the lane's keys in order; every lane of the warp
  // comes along (a lane past the part's end with a kept key)
  auto each = [&](auto&& f) {
    if constexpr (kPer > 0) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (begin + 32 * j >= end) break;
        const int i = begin + 32 * j + lane;
        f(held[j], i);
      }
    } else {
      for (int i0 = begin; i0 < end; i0 += 32) {
        const int i = i0 + lane;
        f(i < end ? keys[i] : kKeptKey, i);
      }
    }
  };
  // the range of the keys that are scores; a kept key + 1 is 0
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
  each([&](uint32_t k, int) {
    lo = min(lo, k);
    hi = max(hi, k + 1);
  });
  lo = __reduce_min_sync(~0u, lo);
  hi = __reduce_max_sync(~0u, hi);
  if (lane == 0) s_lo[warp] = lo, s_hi[warp] = hi;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kTopkWarps; ++w) {
    lo = min(lo, s_lo[w]);
    hi = max(hi, s_hi[w]);
  }
  --hi;
  int need = K - p.kept;  // n > K, and the kept blocks are K at most
  // Selected: the kept keys, those above the range [lo, lo + 2^bits), and the
  // first `need` of those inside.  (need = 0, all kept: none inside.)
  int bits = hi > lo ? 32 - __clz(hi - lo) : 0;
  uint32_t top = hi;  // keys above are taken whole
  if (need > 0) {
    while (bits > 0) {
      const int shift = max(0, bits - kTopkBits);
#pragma unroll
      for (int i = 0; i < kTopkOwn; ++i) hist[tid + i * kTopkThreads] = 0;
      __syncthreads();
      each([&](uint32_t k, int) {
        if (k - lo <= top - lo) atomicAdd(&hist[(k - lo) >> shift], 1);
      });
      __syncthreads();
      // keys in the bins above this thread's
      int own = 0;
#pragma unroll
      for (int i = 0; i < kTopkOwn; ++i) own += hist[kTopkOwn * tid + i];
      int above = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_down_sync(~0u, above, d);
        if (lane + d < 32) above += o;
      }
      if (lane == 0) s_warp[warp] = above;
      __syncthreads();
      above -= own;
      for (int w = warp + 1; w < kTopkWarps; ++w) above += s_warp[w];
      if (above < need && above + own >= need) {
        int bin = kTopkOwn * tid + kTopkOwn - 1;
        for (; above + hist[bin] < need; --bin) above += hist[bin];
        s_bin = bin;
        s_need = need - above;
        s_count = hist[bin];
      }
      __syncthreads();
      lo += (uint32_t)s_bin << shift;
      // (a difference: with a NaN's key in the range, lo + 2^shift may pass 2^32)
      top = lo + min(top - lo, (uint32_t)((1ull << shift) - 1));
      need = s_need;
      bits = shift;
      if (s_count == need) break;  // all of the bin
      __syncthreads();  // hist and s_* are written again
    }
  }
  // in order: the keys above, and the first `need` of those inside
  if (need == 0) lo = 0xFFFFFFFEu, top = 0xFFFFFFFEu;  // the kept keys alone
  int above = 0, equal = 0;
  each([&](uint32_t k, int) {
    above += k > top;
    equal += k - lo <= top - lo;
  });
  // (the lanes past the part's end had kept keys)
  above = __reduce_add_sync(~0u, above) - (((end - begin + 31) & ~31) - (end - begin));
  equal = __reduce_add_sync(~0u, equal);
  __syncthreads();  // s_warp was read above
  if (lane == 0) s_warp[warp] = above, s_equal[warp] = equal;
  __syncthreads();
  int at = 0, eq = 0;  // entries before this warp's part
  for (int w = 0; w < warp; ++w) {
    at += s_warp[w];
    eq += s_equal[w];
  }
  at += min(eq, need);
  const unsigned below = (1u << lane) - 1;
  each([&](uint32_t k, int i) {
    bool take = k > top && i < end;
    const unsigned ge = __ballot_sync(~0u, k - lo <= top - lo);
    if (ge) {  // keys inside: few
      take |= (ge >> lane & 1) && eq + __popc(ge & below) < need;
      eq += __popc(ge);
    }
    const unsigned taken = __ballot_sync(~0u, take);
    if (take) out[at + __popc(taken & below)] = i;
    at += __popc(taken);
  });
}

template <int kPg, int kD>
cudaError_t launch_summarise_d(const StepView& s, const void* k_cache, int num_kv_heads,
                               void* bounds, cudaStream_t stream) {
  // blocks a request of max_query_len tokens writes to, at most
  const int64_t wide = std::min(((int64_t)s.max_query_len + kBS - 2) / kBS + 1,
                                ((int64_t)s.max_seq_len + kBS - 1) / kBS);
  // a warp per KV head, eight to a CTA at most
  const int warps = std::min(num_kv_heads, kThreads / 32);
  const dim3 grid((unsigned)wide, (unsigned)std::min(s.num_seqs, 65535),
                  (unsigned)((num_kv_heads + warps - 1) / warps));
  if (grid.z > 65535) return cudaErrorInvalidValue;
  summarise_kernel<kPg, kD><<<grid, warps * 32, 0, stream>>>(
      s, k_cache, num_kv_heads, static_cast<uint8_t*>(bounds));
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

template <typename TQ, int kD, bool kFew>
cudaError_t launch_score_g(const ScoreParams& p, dim3 grid, cudaStream_t stream) {
  constexpr int kSmem = ScoreLayout<kD>::kSmem;
  const cudaError_t a = cudaFuncSetAttribute(
      score_kernel<TQ, kD, kFew>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (a != cudaSuccess) return a;
  score_kernel<TQ, kD, kFew><<<grid, kScoreWarps * 32, kSmem, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename TQ, int kD>
cudaError_t launch_score_d(const ScoreParams& p, dim3 grid, cudaStream_t stream) {
  return p.group <= kScoreHeads / 2 ? launch_score_g<TQ, kD, true>(p, grid, stream)
                                    : launch_score_g<TQ, kD, false>(p, grid, stream);
}

template <typename TQ>
cudaError_t launch_score(const ScoreParams& p, int head_dim, dim3 grid,
                         cudaStream_t stream) {
  return head_dim == 128 ? launch_score_d<TQ, 128>(p, grid, stream)
                         : launch_score_d<TQ, 64>(p, grid, stream);
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
  pl.pass_tokens = std::max<int64_t>(1, std::min(pl.pass_tokens, kSelectPassTokens));
  pl.pass_tokens = std::min(pl.pass_tokens, num_tokens);
  // What is asked for grows with every size, so that a buffer for a loop's longest
  // step holds every shorter one: of a step in passes, the whole bound, not the
  // tokens of a pass times their bytes.
  pl.bytes = std::min(std::min<int64_t>(num_tokens, kSelectPassTokens) * token_bytes,
                      std::max(kSelectScoreBytes, token_bytes));
  return pl;
}

cudaError_t launch_select_blocks(const StepView& s, const SelectPlan& plan,
                                 const void* q, pa_dtype q_dtype, int num_q_heads,
                                 int num_kv_heads, int head_dim, const void* bounds,
                                 int max_selected, int keep_first, int keep_last,
                                 int32_t* selected, int32_t* num_selected,
                                 void* workspace, int num_sms, cudaStream_t stream) {
  const int max_blocks = (int)(((int64_t)s.max_seq_len + kBS - 1) / kBS);
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
      // as many blocks per CTA as leave four CTAs per SM: a warp's work on the
      // query (its codes) is then spread over more records
      const int64_t heads = (num_kv_heads + kScoreWarps - 1) / kScoreWarps;
      if (heads > 65535) return cudaErrorInvalidValue;
      p.chunk = kScoreChunkMax * std::max(1, kScoreWarps / num_kv_heads);
      while (p.chunk > kScoreChunkMin &&
             nt * heads * ((max_blocks + p.chunk - 1) / p.chunk) < 4ll * num_sms)
        p.chunk /= 2;
      const dim3 grid((unsigned)((max_blocks + p.chunk - 1) / p.chunk), (unsigned)nt,
                      (unsigned)heads);
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
    tp.kept = keep_first + keep_last;
    tp.row_scores = plan.row_scores;
    tp.keys = static_cast<const uint32_t*>(workspace);
    tp.selected = selected;
    tp.num_selected = num_selected;
    if (nt * num_kv_heads > 0x7fffffffll) return cudaErrorInvalidValue;
    // starts while the scores are being made, waits for them
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(nt * num_kv_heads));
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = max_blocks > max_selected ? 1 : 0;
    // 256 threads to a row where there are rows enough for every SM (four to an
    // SM: 512 rows of 512 to 4096 blocks 10 us, with 512 threads a quarter more) or
    // few blocks (both kernels, 8 rows of 512 blocks: 8.4 us, with 1024 threads
    // 10.0; 32 rows of 2048: 10.5 and 11.5); else 1024 (8 rows of 8192: 13.7 us,
    // with 256 14.6).  A row's keys stay in registers up to 8192 blocks, or 16384
    // by 1024 threads (8 rows of those: 23.2 us, read again each time 27.2).
    const bool narrow = nt * num_kv_heads > num_sms || max_blocks <= 16 * 256;
    cfg.blockDim = dim3(narrow ? 256 : 1024);
    const cudaError_t e =
        !narrow ? (max_blocks <= 8 * 1024    ? cudaLaunchKernelEx(&cfg, topk_kernel<1024, 8>, tp)
                   : max_blocks <= 16 * 1024 ? cudaLaunchKernelEx(&cfg, topk_kernel<1024, 16>, tp)
                                             : cudaLaunchKernelEx(&cfg, topk_kernel<1024, 0>, tp))
        : max_blocks <= 4 * 256  ? cudaLaunchKernelEx(&cfg, topk_kernel<256, 4>, tp)
        : max_blocks <= 16 * 256 ? cudaLaunchKernelEx(&cfg, topk_kernel<256, 16>, tp)
        : max_blocks <= 32 * 256 ? cudaLaunchKernelEx(&cfg, topk_kernel<256, 32>, tp)
                                 : cudaLaunchKernelEx(&cfg, topk_kernel<256, 0>, tp);
    if (e != cudaSuccess) return e;
    count_launch();
  }
  return cudaSuccess;
}

}  // namespace pa
