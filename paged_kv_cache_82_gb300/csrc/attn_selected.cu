// attn_selected.cu -- attention of each token over a list of its cache blocks
// (pa_attention_selected).
//
//   out = sum_j softmax(scale <q, k_j>)_j v_j  over the keys j of the listed
//   blocks up to the token's own position; a list of no blocks gives zeros.
//
// A row is one (token, KV head) with its list; all rows' list entries, end to
// end and with a few units for each row's start, are cut into equal shares, one
// CTA each, as many as are resident (every CTA sums the rows' list lengths for
// itself).  A share holds whole
// lists and, at its ends, parts of lists; a second kernel joins those, part by
// part in order.  So a few long lists and many short ones both keep every SM
// busy to the end.
//
// A row reads each listed block's K and V page once and does 4 G multiply-
// adds per element read (G query heads): far below the tensor cores' rate, so
// it is bound by HBM and the pages' latency.  Pages go from HBM straight into
// the registers that feed the MMAs: with the keys as the rows of the first
// product (S^T = K Q^T) and the channels as the rows of the second (O^T = V^T
// P^T), a lane's 16-byte loads are its operand words -- the order of the
// channels inside a product is free, so the lane's 8 (or 16) consecutive
// channels take the places its MMA operand wants.  No shared memory, no
// barrier in the loop: each warp walks its own pages, and the next page's K
// (then V) loads go out as soon as the MMAs have consumed the registers.
//
// 64 tokens x 8 KV heads x 128 blocks of 128 channels, 4 query heads each: bf16 89
// us, 6.0 TB/s (90 % of a copy); 32 x 8 x 256 blocks of E4M3, 8 heads: 56 us, 4.8
// TB/s.  About 12 us of either are the way to the first page (list lengths,
// request, block id, page: four dependent loads) and the join.  One token: 9.3 us.
#include <algorithm>

#include "pa_step.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kJoinThreads = 256;  // 8 heads x 128 channels, four per thread
// A share's units: a row's list entries, and kRowCost for what a CTA needs to
// begin a row (its lookups and the first pages' latency, about 4 us: as long as
// 8 pages of its 4 warps take).  56 rows of 1 to 57 blocks: 9.6 us, without it 28
// (short rows strung together).  Shares have kMinShare units at least, two pages
// per warp: one row's 128 blocks 11 to 12 us with 8 or 16, 14 with 4 or 32.
constexpr int kRowCost = 8;
constexpr int kMinShare = 8;
constexpr float kLog2e = 1.4426950408889634f;

enum : int { kB16 = 0, kH16, kF8, kI4, kN4, kF32 };  // bf16, f16, E4M3, INT4, NVFP4, fp32 pages

struct SelParams {
  StepView s;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  int num_q_heads, num_kv_heads, group;
  int head_rows;  // query heads of a KV head that one CTA takes (grid.y: parts)
  const int32_t* selected;
  const int32_t* num_selected;
  int max_selected;
  float scale, k_scale, v_scale;
  void* out;
  // parts of lists, two per CTA: 0 of a list that began in a CTA before, 1 of
  // one that begins here and goes on
  float* part;     // [CTA][2][head_rows][D]
  float* part_ml;  // [CTA][2][head_rows][2]: m, l
  int2* cut;       // [CTA]: the row whose list goes on (-1: none), its parts
};

// A row: its token, request, position and list length (-1: the token belongs
// to no request, or its metadata is broken, which check_requests flags).
struct Unit {
  int64_t t;
  int h;
  int r, pos, count;
};

__device__ __forceinline__ Unit find_unit(const SelParams& p, int64_t row, bool tell) {
  Unit u;
  u.t = row / p.num_kv_heads;
  u.h = (int)(row - u.t * p.num_kv_heads);
  u.count = __ldg(p.num_selected + row);
  const TokenReq q = warp_token_request(
      p.s.query_start_loc, p.s.seq_lens, p.s.num_seqs, u.t, p.s.num_tokens,
      p.s.max_query_len, p.s.max_seq_len, p.s.max_blocks_per_seq);
  u.r = q.r;
  u.pos = q.m.L - q.m.n + (int)(u.t - q.m.q0);
  if (!q.in || !q.m.ok) {
    u.count = -1;
  } else if (u.count < 0 || u.count > p.max_selected) {
    if (tell) flag_error(p.s.err, PA_DEV_ERR_METADATA);
    u.count = 0;
  }
  return u;
}

// Entry i of a row's list as it is there, and the one before it: read without
// the row's request, on their way while that is looked up.
struct Listed {
  int block, before;
};
__device__ __forceinline__ Listed listed(const SelParams& p, int64_t row, int i) {
  const int32_t* list = p.selected + row * p.max_selected;
  return Listed{__ldg(list + i), i > 0 ? __ldg(list + i - 1) : -1};
}

// The logical block and its physical block (-1: skipped, with a flag -- not
// above the entry before it, past the token's position, or a bad physical id).
struct Entry {
  int block, phys;
};
__device__ __forceinline__ Entry list_entry(const SelParams& p, const Unit& u,
                                            const Listed& at) {
  Entry e{at.block, -1};
  if (e.block <= at.before || e.block < 0 || e.block > u.pos / kBS) {
    flag_error(p.s.err, PA_DEV_ERR_METADATA);
    return e;
  }
  const int b =
      __ldg(p.s.block_tables + (int64_t)u.r * p.s.max_blocks_per_seq + e.block);
  if (b < 0 || (int64_t)b >= p.s.num_blocks)
    flag_error(p.s.err, PA_DEV_ERR_BLOCK_ID);
  else
    e.phys = b;
  return e;
}

// 2^x to 2 units in the last place of fp32; below 2^-126: 0
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// x as the sum of two bf16 numbers: its upper half, and what that leaves, rounded;
// together off by 2^-16 of x.  Cut off and not rounded, the head leaves a tail of
// x's sign.  kPositive, x >= 0: the tail is 2^-126 at least and not 0, so that both
// times an infinite value are the same infinity.
__device__ __forceinline__ uint32_t bf16_heads(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
template <bool kPositive>
__device__ __forceinline__ float bf16_tail(float x) {
  const float tail = x - __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
  return kPositive ? fmaxf(tail, 0x1p-126f) : tail;
}

template <int kPg, int kD>
struct PageTraits {
  static constexpr bool k4 = kPg == kI4 || kPg == kN4;
  static constexpr int kRowBytes = k4 ? kD / 2 : kPg == kF8 ? kD : 2 * kD;  // codes
  static constexpr int kPageBytes = kPg == kI4   ? PA_PAGE_BYTES(PA_INT4, kD)
                                    : kPg == kN4 ? PA_PAGE_BYTES(PA_NVFP4, kD)
                                                 : kBS * kRowBytes;
  // K: lane (r, c) reads kKBytes at kKBytes c + 4 kKBytes i of rows r and r + 8
  static constexpr int kKBytes = kRowBytes >= 64 ? 16 : kRowBytes / 4;
  static constexpr int kKChunks = kRowBytes / (4 * kKBytes);
  // V: lane (r, c) reads kVBytes at kVBytes r + 8 kVBytes i of the rows 2c, 2c +
  // 1, 2c + 8, 2c + 9
  static constexpr int kVBytes = kRowBytes >= 128 ? 16 : kRowBytes / 8;
  static constexpr int kVChunks = kRowBytes / (8 * kVBytes);
  static constexpr int kTiles = kD / 16;  // m16 tiles of the output's channels
  // channels of a lane's K chunk
  static constexpr int kKChannels = kD / (4 * kKChunks);
  // The products' types: Q K in the 16-bit type of the pages, in f16 over the
  // others; P V as well, over INT4 pages in bf16 (their scales are in P, which
  // then needs that range).  P is one f16 number (11 bits: off by 2^-11 of it), or
  // two bf16 numbers: one has 8 bits, and two keys' average was off by 5e-3, where
  // pa_attention is within 2e-3.  The second MMA per tile costs little beside the
  // pages: 64 tokens x 8 heads x 128 blocks 89.2 us, with one part 88.7.
  static constexpr bool kQkBF = kPg == kB16;
  static constexpr bool kPvBF = kPg == kB16 || kPg == kI4;
  // NVFP4 values are decoded 2^-7 of their size, so that code and scale stay
  // within f16 on the way
  static constexpr float kUnit = kPg == kN4 ? 128.f : 1.f;
  // Pages of one step: 8 KB of K and V in a warp's registers, whatever the
  // type, are on their way while the step before is computed (4-bit pages,
  // bound by their decoding: two).  FP8, 32 tokens x 8 heads x 256 blocks: 57 us
  // with two pages, 76 with one.
  static constexpr int kPages = k4 ? 2 : 4096 / (kBS * kRowBytes);
};

// kBytes (4, 8 or 16) as words
template <int kBytes>
__device__ __forceinline__ void load_words(uint32_t* w, const uint8_t* src) {
  if constexpr (kBytes == 16) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(src));
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else if constexpr (kBytes == 8) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(src));
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
  }
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Nibble k of each 16-bit half of x, an INT4 code, as a pair: in f16 from 1024 +
// (code + 8), in bf16 from 128 + (code + 8), both exact.
template <bool kBF, int k>
__device__ __forceinline__ uint32_t int4_pair(uint32_t x) {
  const uint32_t u = ((x >> (4 * k)) & 0x000F000Fu) ^ (kBF ? 0x43084308u : 0x64086408u);
  uint32_t d;
  if constexpr (kBF)
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(u), "r"(0x43084308u));
  else
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(u), "r"(0x64086408u));
  return d;
}

// Nibble k of each half, an E2M1 code, as an f16 pair 2^-14 of its size: sign,
// two exponent bits and the mantissa bit where f16 has its own lowest ones.
template <int k>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t x) {
  const uint32_t sign = k == 3 ? x : x << (12 - 4 * k);
  const uint32_t mag = k == 3 ? x >> 3 : x << (k == 3 ? 0 : 9 - 4 * k);
  return (sign & 0x80008000u) | (mag & 0x0E000E00u);
}

// 128 times the values of two E4M3 bytes, as f16; at most 57344
__device__ __forceinline__ uint32_t e4m3_pair_128(uint32_t bytes) {
  uint32_t d;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(d)
      : "r"(bytes));
  return mul_f16x2(d, 0x58005800u);
}

// CTAs per SM that the kernels are built for: what the accumulators of 8 or 16
// query heads, or a warp's fp32 pages (128 registers), leave of the registers
constexpr int ctas_per_sm(bool fp32, int head_rows) {
  return !fp32 && head_rows == 8 ? 3 : 2;
}

// Entries of a row's list that count: none of a row past the last request.
__device__ __forceinline__ int list_length(const SelParams& p, int64_t row) {
  const int c = __ldg(p.num_selected + row);
  return c > 0 && c <= p.max_selected ? c : 0;
}

// A CTA's share of all the rows' units (a row's kRowCost come first).
struct Share {
  int64_t begin, end;
  int64_t size;        // of every share
  int64_t row;         // the row that `begin` lies in,
  int64_t row_begin;   // and where its entries begin
};

__device__ __forceinline__ int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

// Every thread sums a contiguous part of the rows; the one whose part holds
// the share's first unit walks it.  Its first counts go out together with the
// last request's end, which bounds the rows (*rows).
__device__ __forceinline__ Share find_share(const SelParams& p, int64_t* rows) {
  constexpr int kHeld = 4;
  __shared__ int64_t warp_sums[32], total, s_row, s_row_begin;
  const int64_t all = p.s.num_tokens * p.num_kv_heads;
  const int64_t part = (all + kThreads - 1) / kThreads;
  const int64_t lo = least(all, threadIdx.x * part), hi = least(all, lo + part);
  int held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    held[k] = lo + k < hi ? __ldg(p.num_selected + lo + k) : 0;
  const int64_t last = __ldg(p.s.query_start_loc + p.s.num_seqs);
  // (an end before the first token is broken metadata: each row looks for itself)
  *rows = (last < 0 ? p.s.num_tokens : least(last, p.s.num_tokens)) * p.num_kv_heads;
  const int64_t end = least(hi, *rows);
  auto units = [&](int count) {
    return count > 0 && count <= p.max_selected ? count + kRowCost : 0;
  };
  int64_t sum = 0;
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (lo + k < end) sum += units(held[k]);
  for (int64_t i = lo + kHeld; i < end; ++i) sum += units(__ldg(p.num_selected + i));
  const int64_t before = block_scan_excl(sum, &total, warp_sums);
  Share s;
  s.size = (total + gridDim.x - 1) / gridDim.x;
  if (s.size < kMinShare) s.size = kMinShare;
  s.begin = least(total, blockIdx.x * s.size);
  s.end = least(total, s.begin + s.size);
  if (s.begin < s.end && s.begin >= before && s.begin < before + sum) {
    int64_t at = before, i = lo;
    for (int c; at + (c = units(__ldg(p.num_selected + i))) <= s.begin; ++i) at += c;
    s_row = i;
    s_row_begin = at + kRowCost;
  }
  __syncthreads();
  s.row = s_row;
  s.row_begin = s_row_begin;
  return s;
}

template <typename TQ, int kPg, int kD, int kRows>
__device__ __forceinline__ bool attend_part(const SelParams& p, int64_t row, int begin,
                                            int end, int slot);
template <int kD, int kRows>
__device__ __forceinline__ bool attend_part_f32(const SelParams& p, int64_t row, int begin,
                                                int end, int slot);

template <typename TQ, int kPg, int kD, int kRows>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(kPg == kF32, kRows))
selected_kernel(const SelParams p) {
  pdl_launch_dependents();
  int64_t rows;  // of tokens up to the last request's
  const Share sh = find_share(p, &rows);
  const int cta = blockIdx.y * gridDim.x + blockIdx.x;
  int2 cut = make_int2(-1, 0);
  int64_t row = sh.row, row_begin = sh.row_begin;
  if (sh.begin < sh.end) {
    while (row_begin < sh.end) {
      const int64_t row_end = row_begin + list_length(p, row);
      const int64_t begin = row_begin < sh.begin ? sh.begin : row_begin;
      const int64_t end = least(row_end, sh.end);
      // -1: the whole list is here; else the CTA's place for a part
      const int slot = begin == row_begin && end == row_end ? -1 : begin > row_begin ? 0 : 1;
      const int from = (int)(begin - row_begin), to = (int)(end - row_begin);
      bool done;
      if constexpr (kPg == kF32)
        done = attend_part_f32<kD, kRows>(p, row, from, to, slot);
      else
        done = attend_part<TQ, kPg, kD, kRows>(p, row, from, to, slot);
      if (done && slot == 1)
        cut = make_int2((int)row, (int)((row_end - 1) / sh.size - blockIdx.x + 1));
      // the next row with a list
      do {
        if (++row >= rows) break;
      } while (list_length(p, row) == 0);
      if (row >= rows) break;
      row_begin = row_end + kRowCost;
    }
  }
  if (threadIdx.x == 0) p.cut[cta] = cut;
}

// The four warps' results in shared memory -- m, l and the sum of the values
// for each of the CTA's query heads -- as one: to the output if that is all of
// the list (slot < 0), else to the CTA's place for a part.
template <typename TQ, int kRows, int kD>
__device__ __forceinline__ void finish_part(const SelParams& p, const Unit& u, int slot,
                                            float unit,
                                            const float (&s_acc)[kWarps][kRows][kD],
                                            const float (&s_m)[kWarps][kRows],
                                            const float (&s_l)[kWarps][kRows]) {
  const int heads = min(p.group - (int)blockIdx.y * kRows, kRows);
  const int head0 = u.h * p.group + blockIdx.y * kRows;
  __syncthreads();
  for (int i = threadIdx.x; i < heads * kD; i += kThreads) {
    const int hd = i / kD, d = i - hd * kD;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][hd]);
    float a = 0.f, ls = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = s_m[w][hd] == -INFINITY ? 0.f : exp2f(s_m[w][hd] - mx);
      a += f * s_acc[w][hd][d];
      ls += f * s_l[w][hd];
    }
    a *= unit;
    if (slot < 0) {
      static_cast<TQ*>(p.out)[(u.t * p.num_q_heads + head0 + hd) * kD + d] =
          from_f32<TQ>(ls == 0.f ? 0.f : a / ls * p.v_scale);
    } else {
      const int64_t at =
          ((int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * 2 + slot) * p.head_rows + hd;
      p.part[at * kD + d] = a;
      if (d == 0) {
        p.part_ml[2 * at] = mx;
        p.part_ml[2 * at + 1] = ls;
      }
    }
  }
  __syncthreads();  // the next part writes the shared memory again
}

// Entries begin .. end - 1 of a row's list, by the tensor cores.  False: the row
// is no request's, or its metadata is broken.
template <typename TQ, int kPg, int kD, int kRows>
__device__ __forceinline__ bool attend_part(const SelParams& p, int64_t row, int begin,
                                            int end, int slot) {
  using Tr = PageTraits<kPg, kD>;
  constexpr bool kScaled = Tr::k4;  // pages with scales of their own
  constexpr int kNT = kRows / 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, c = lane & 3;
  constexpr int kP = Tr::kPages;
  // The warp's steps: kP entries in a row from begin + kP warp, then kP kWarps
  // further on.  The lanes hold the next 32 of the warp's entries.
  const int first = begin + kP * warp;
  const int steps = end > first ? (end - first + kP * kWarps - 1) / (kP * kWarps) : 0;
  auto place = [&](int i) { return first + (i / kP) * (kP * kWarps) + i % kP; };
  Listed ahead{0, 0};
  if (place(lane) < end) ahead = listed(p, row, place(lane));
  const Unit u = find_unit(p, row, threadIdx.x == 0);
  if (u.count <= 0) return false;
  const int part = blockIdx.y;
  const int heads = min(p.group - part * kRows, kRows);
  const int head0 = u.h * p.group + part * kRows;

  float acc[kNT][Tr::kTiles][4];
  float m[kNT][2], l[kNT][2];
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
    for (int i = 0; i < Tr::kTiles; ++i)
      acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
  }

  constexpr int kKW = Tr::kKBytes / 4, kVW = Tr::kVBytes / 4;
  uint32_t kr[kP][2][Tr::kKChunks][kKW];
  uint32_t vr[kP][4][Tr::kVChunks][kVW];
  // 4-bit pages: INT4, the scales of keys r and r + 8 (fp32); NVFP4, E4M3 scales
  // of K rows r and r + 8 (the lane's blocks) and of the four V rows (its block)
  uint32_t ks[kP][2], vs[kP][kPg == kN4 ? 4 : 2];
  constexpr int64_t kPageBytes = Tr::kPageBytes;
  const uint8_t* kbase = static_cast<const uint8_t*>(p.k_cache) + (int64_t)u.h * kPageBytes;
  const uint8_t* vbase = static_cast<const uint8_t*>(p.v_cache) + (int64_t)u.h * kPageBytes;
  const int64_t block_bytes = kPageBytes * p.num_kv_heads;
  constexpr int kScales = kBS * Tr::kRowBytes;  // where they begin

  // keys of a page up to the token's position
  auto page_keys = [&](const Entry& e) {
    return e.phys < 0 ? 0 : min(kBS, u.pos - e.block * kBS + 1);
  };
  // Loads are unconditional: a skipped entry reads block 0, rows past the
  // position what happens to be there.  The few steps with such keys mask them
  // where they are used.
  auto load_k = [&](const Entry (&en)[kP]) {
#pragma unroll
    for (int g = 0; g < kP; ++g) {
      const uint8_t* page = kbase + (int64_t)max(en[g].phys, 0) * block_bytes;
#pragma unroll
      for (int i = 0; i < Tr::kKChunks; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          load_words<Tr::kKBytes>(kr[g][j][i], page + (r + 8 * j) * Tr::kRowBytes +
                                                   (c + 4 * i) * Tr::kKBytes);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (kPg == kI4)
          ks[g][j] = __ldg(reinterpret_cast<const uint32_t*>(page + kScales) + r + 8 * j);
        else if constexpr (kPg == kN4 && kD == 128)
          ks[g][j] = __ldg(reinterpret_cast<const uint16_t*>(page + kScales) + (r + 8 * j) * 4 + c);
        else if constexpr (kPg == kN4)
          ks[g][j] = __ldg(page + kScales + (r + 8 * j) * 4 + c);
      }
    }
  };
  auto load_v = [&](const Entry (&en)[kP]) {
#pragma unroll
    for (int g = 0; g < kP; ++g) {
      const uint8_t* page = vbase + (int64_t)max(en[g].phys, 0) * block_bytes;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = 2 * c + (j & 1) + 8 * (j >> 1);
#pragma unroll
        for (int i = 0; i < Tr::kVChunks; ++i)
          load_words<Tr::kVBytes>(vr[g][j][i],
                                  page + key * Tr::kRowBytes + (r + 8 * i) * Tr::kVBytes);
        if constexpr (kPg == kN4)
          vs[g][j] = __ldg(page + kScales + key * (kD / 16) + (kD == 128 ? r : r / 2));
      }
      if constexpr (kPg == kI4) {
        vs[g][0] = __ldg(reinterpret_cast<const uint32_t*>(page + kScales) + r);
        vs[g][1] = __ldg(reinterpret_cast<const uint32_t*>(page + kScales) + r + 8);
      }
    }
  };

  Entry held{0, -1};
  auto entries = [&](int step, Entry (&en)[kP]) {
    const int i = step * kP;  // of the warp's entries
    if ((i & 31) == 0) {
      const int at = place(i + lane);
      held = Entry{0, -1};
      if (at < end) held = list_entry(p, u, i == 0 ? ahead : listed(p, row, at));
    }
#pragma unroll
    for (int g = 0; g < kP; ++g)
      en[g] = Entry{__shfl_sync(~0u, held.block, (i & 31) + g),
                    __shfl_sync(~0u, held.phys, (i & 31) + g)};
  };
  Entry cur[kP];
  if (steps > 0) {
    entries(0, cur);
    load_k(cur);
    load_v(cur);
  }

  // Q operand words, in the channel order of the lane's K words: neighbours,
  // over INT4 pages the channels 4 apart that a mask leaves in one word.  Where
  // the products are in f16 over a narrower page, a power of two of each head's own
  // brings its largest query to 2^13, well inside f16's range either way, and leaves
  // through the score's scale (that of the heads 2c, 2c + 1 of the scores here).
  constexpr int kE = Tr::kKChannels;
  constexpr bool kHeadScale = kPg == kF8 || kScaled;
  uint32_t qw[kNT][Tr::kKChunks][kE / 2];
  float score_scale[kHeadScale ? kNT : 1][kHeadScale ? 2 : 1];
  {
    // a scale of either sign, or 0: the score's stays positive
    const float scale = p.scale * p.k_scale * (Tr::kUnit * kLog2e);
    const float sign = scale > 0.f ? 1.f : scale < 0.f ? -1.f : 0.f;
    score_scale[0][0] = scale == 0.f ? 1.f : fabsf(scale);
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const int hd = nt * 8 + r;
      float x[Tr::kKChunks][kE], down = sign;
      float big = 0.f;  // the largest finite one
#pragma unroll
      for (int i = 0; i < Tr::kKChunks; ++i) {
        const TQ* src = static_cast<const TQ*>(p.q) +
                        (u.t * p.num_q_heads + head0 + hd) * kD + (c + 4 * i) * kE;
        uint4 w[kE / 8];
#pragma unroll
        for (int e = 0; e < kE / 8; ++e)
          w[e] = hd < heads ? __ldg(reinterpret_cast<const uint4*>(src) + e)
                            : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          x[i][e] = to_f32(reinterpret_cast<const TQ*>(w)[e]);
          if constexpr (kHeadScale)
            if (fabsf(x[i][e]) < INFINITY) big = fmaxf(big, fabsf(x[i][e]));
        }
      }
      if constexpr (kHeadScale) {
        big = fmaxf(big, __shfl_xor_sync(~0u, big, 1));
        big = fmaxf(big, __shfl_xor_sync(~0u, big, 2));
        // (2^120 and a bf16 query of 2^-133 are a normal f16 number as well)
        const int ex = big > 0.f ? max(ilogbf(big) - 13, -120) : 0;
        down *= exp2f((float)-ex);
        const float up = fabsf(scale == 0.f ? 1.f : scale) * exp2f((float)ex);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          score_scale[nt][j] = __shfl_sync(~0u, up, (2 * c + j) * 4);
      }
#pragma unroll
      for (int i = 0; i < Tr::kKChunks; ++i)
#pragma unroll
        for (int w = 0; w < kE / 2; ++w) {
          const int e0 = kPg == kI4 ? 8 * (w / 4) + w % 4 : 2 * w;
          const int e1 = kPg == kI4 ? e0 + 4 : e0 + 1;
          qw[nt][i][w] = pack2<Tr::kQkBF>(x[i][e0] * down, x[i][e1] * down);
        }
    }
  }

  for (int i = 0; i < steps; ++i) {
    // S^T = K Q^T: keys r and r + 8, heads 2c and 2c + 1
    float s[kP][kNT][4];
#pragma unroll
    for (int g = 0; g < kP; ++g) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
        s[g][nt][0] = s[g][nt][1] = s[g][nt][2] = s[g][nt][3] = 0.f;
#pragma unroll
      for (int ch = 0; ch < Tr::kKChunks; ++ch) {
        const uint32_t(&w0)[kKW] = kr[g][0][ch];
        const uint32_t(&w1)[kKW] = kr[g][1][ch];
        // operand words of a lane's channels, a step's two (per row) at a time
        auto product = [&](uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, int w) {
          const uint32_t a[4] = {a0, a1, a2, a3};
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
            mma16816<Tr::kQkBF>(s[g][nt], a, qw[nt][ch][w], qw[nt][ch][w + 1]);
        };
        if constexpr (kPg == kB16 || kPg == kH16) {
#pragma unroll
          for (int w = 0; w < kKW; w += 2) product(w0[w], w1[w], w0[w + 1], w1[w + 1], w);
        } else if constexpr (kPg == kF8) {
#pragma unroll
          for (int w = 0; w < kKW; ++w) {
            uint32_t a[4];
            e4m3x4_to_f16x2x2(w0[w], a[0], a[2]);
            e4m3x4_to_f16x2x2(w1[w], a[1], a[3]);
            product(a[0], a[1], a[2], a[3], 2 * w);
          }
        } else if constexpr (kPg == kI4) {
#pragma unroll
          for (int w = 0; w < kKW; ++w) {
            product(int4_pair<false, 0>(w0[w]), int4_pair<false, 0>(w1[w]),
                    int4_pair<false, 1>(w0[w]), int4_pair<false, 1>(w1[w]), 4 * w);
            product(int4_pair<false, 2>(w0[w]), int4_pair<false, 2>(w1[w]),
                    int4_pair<false, 3>(w0[w]), int4_pair<false, 3>(w1[w]), 4 * w + 2);
          }
        } else {
#pragma unroll
          for (int w = 0; w < kKW; ++w) {
            // two words are a block of 16 channels
            const uint32_t s0 = e4m3_pair_128(((ks[g][0] >> (8 * (w / 2))) & 0xFFu) * 0x0101u);
            const uint32_t s1 = e4m3_pair_128(((ks[g][1] >> (8 * (w / 2))) & 0xFFu) * 0x0101u);
            // halves (byte i, byte i + 2) -> neighbours: bytes 0, 1 and 2, 3
            const uint32_t l0 = __byte_perm(w0[w], 0, 0x4140), h0 = __byte_perm(w0[w], 0, 0x4342);
            const uint32_t l1 = __byte_perm(w1[w], 0, 0x4140), h1 = __byte_perm(w1[w], 0, 0x4342);
            // l: byte 0 in the low half, byte 1 in the high one; nibbles 0 and 1
            // of a half are neighbours
            auto near = [](uint32_t even, uint32_t odd, bool up) {
              return __byte_perm(even, odd, up ? 0x7632 : 0x5410);
            };
            const uint32_t a0 = e2m1_pair<0>(l0), a1 = e2m1_pair<1>(l0);
            const uint32_t b0 = e2m1_pair<0>(h0), b1 = e2m1_pair<1>(h0);
            const uint32_t c0 = e2m1_pair<0>(l1), c1 = e2m1_pair<1>(l1);
            const uint32_t d0 = e2m1_pair<0>(h1), d1 = e2m1_pair<1>(h1);
            product(mul_f16x2(near(a0, a1, false), s0), mul_f16x2(near(c0, c1, false), s1),
                    mul_f16x2(near(a0, a1, true), s0), mul_f16x2(near(c0, c1, true), s1),
                    4 * w);
            product(mul_f16x2(near(b0, b1, false), s0), mul_f16x2(near(d0, d1, false), s1),
                    mul_f16x2(near(b0, b1, true), s0), mul_f16x2(near(d0, d1, true), s1),
                    4 * w + 2);
          }
        }
      }
      if constexpr (kPg == kI4) {  // the keys' own scales
        const float s0 = __uint_as_float(ks[g][0]), s1 = __uint_as_float(ks[g][1]);
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          s[g][nt][0] *= s0;
          s[g][nt][1] *= s0;
          s[g][nt][2] *= s1;
          s[g][nt][3] *= s1;
        }
      }
    }
    int keys[kP], fewest = kBS;
#pragma unroll
    for (int g = 0; g < kP; ++g) {
      keys[g] = page_keys(cur[g]);
      fewest = min(fewest, keys[g]);
    }
    if (i + 1 < steps) {
      entries(i + 1, cur);
      load_k(cur);
    }
    if (fewest < kBS) {  // masked keys: no score, and no value that could be NaN
#pragma unroll
      for (int g = 0; g < kP; ++g) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (r + 8 * (j >> 1) >= keys[g]) s[g][nt][j] = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (2 * c + (j & 1) + 8 * (j >> 1) >= keys[g])
#pragma unroll
            for (int ch = 0; ch < Tr::kVChunks; ++ch)
#pragma unroll
              for (int w = 0; w < kVW; ++w) vr[g][j][ch][w] = 0;
        if constexpr (kScaled)
#pragma unroll
          for (int j = 0; j < (kPg == kN4 ? 4 : 2); ++j)
            if ((kPg == kN4 ? 2 * c + (j & 1) + 8 * (j >> 1) : r + 8 * j) >= keys[g])
              vs[g][j] = 0;
      }
    }
    // softmax over the step's keys, by scores that are rounded once: in one fma with
    // the maximum the largest one's own exponent would be that rounding and not 0,
    // 2^5 where scores reach 2^30
    uint32_t pb[kP][kNT][2], pl[kP][kNT][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int g = 0; g < kP; ++g)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[g][nt][j] *= score_scale[kHeadScale ? nt : 0][kHeadScale ? j & 1 : 0];
      float mx[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mx[j] = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
#pragma unroll
        for (int g = 1; g < kP; ++g) mx[j] = fmaxf(mx[j], fmaxf(s[g][nt][j], s[g][nt][j + 2]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) mx[j] = fmaxf(mx[j], __shfl_xor_sync(~0u, mx[j], d));
        mx[j] = fmaxf(mx[j], m[nt][j]);
      }
      if (__any_sync(~0u, mx[0] > m[nt][0] || mx[1] > m[nt][1])) {
        float al[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          al[j] = mx[j] == -INFINITY ? 1.f : exp2_fast(m[nt][j] - mx[j]);
          m[nt][j] = mx[j];
          l[nt][j] *= al[j];
        }
#pragma unroll
        for (int tl = 0; tl < Tr::kTiles; ++tl) {
          acc[nt][tl][0] *= al[0];
          acc[nt][tl][1] *= al[1];
          acc[nt][tl][2] *= al[0];
          acc[nt][tl][3] *= al[1];
        }
      }
      const float m0 = m[nt][0] == -INFINITY ? 0.f : -m[nt][0];
      const float m1 = m[nt][1] == -INFINITY ? 0.f : -m[nt][1];
#pragma unroll
      for (int g = 0; g < kP; ++g) {
        const float p0 = exp2_fast(s[g][nt][0] + m0);
        const float p1 = exp2_fast(s[g][nt][1] + m1);
        const float p2 = exp2_fast(s[g][nt][2] + m0);
        const float p3 = exp2_fast(s[g][nt][3] + m1);
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        // keys as rows -> heads as rows: the second product's operand, by bf16
        // products in two parts.  Over INT4 pages the values' scales go into P.
        if constexpr (Tr::kPvBF) {
          float x[4] = {p0, p1, p2, p3}, y[4];
          if constexpr (kPg == kI4) {
            const float s0 = __uint_as_float(vs[g][0]), s1 = __uint_as_float(vs[g][1]);
            x[0] *= s0, x[1] *= s0, x[2] *= s1, x[3] *= s1;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = bf16_tail<kPg == kB16>(x[j]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            pb[g][nt][j] = transpose8x8(bf16_heads(x[2 * j], x[2 * j + 1]));
            pl[g][nt][j] = transpose8x8(pack2<true>(y[2 * j], y[2 * j + 1]));
          }
        } else {
          pb[g][nt][0] = transpose8x8(pack2<false>(p0, p1));
          pb[g][nt][1] = transpose8x8(pack2<false>(p2, p3));
        }
      }
    }
    // O^T += V^T P^T: channels as rows
#pragma unroll
    for (int g = 0; g < kP; ++g)
#pragma unroll
      for (int ch = 0; ch < Tr::kVChunks; ++ch)
#pragma unroll
        for (int w = 0; w < kVW; ++w) {
          const uint32_t a0 = vr[g][0][ch][w], a1 = vr[g][1][ch][w];
          const uint32_t a2 = vr[g][2][ch][w], a3 = vr[g][3][ch][w];
          // tile tl of the lane's channels 2 tl, 2 tl + 1: keys 2c, 2c + 1 of
          // each, then keys 2c + 8, 2c + 9
          auto product = [&](int tl, uint32_t x0, uint32_t x1, uint32_t y0, uint32_t y1) {
            const uint32_t a[4] = {x0, x1, y0, y1};
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
              mma16816<Tr::kPvBF>(acc[nt][tl], a, pb[g][nt][0], pb[g][nt][1]);
              if constexpr (Tr::kPvBF)
                mma16816<true>(acc[nt][tl], a, pl[g][nt][0], pl[g][nt][1]);
            }
          };
          if constexpr (kPg == kB16 || kPg == kH16) {
            product(ch * kVW + w, __byte_perm(a0, a1, 0x5410), __byte_perm(a0, a1, 0x7632),
                    __byte_perm(a2, a3, 0x5410), __byte_perm(a2, a3, 0x7632));
          } else if constexpr (kPg == kF8) {
            // four channels of two keys: bytes of the two rows side by side
            uint32_t x[4], y[4];
            e4m3x4_to_f16x2x2(__byte_perm(a0, a1, 0x5140), x[0], x[1]);
            e4m3x4_to_f16x2x2(__byte_perm(a0, a1, 0x7362), x[2], x[3]);
            e4m3x4_to_f16x2x2(__byte_perm(a2, a3, 0x5140), y[0], y[1]);
            e4m3x4_to_f16x2x2(__byte_perm(a2, a3, 0x7362), y[2], y[3]);
            product((ch * kVW + w) * 2, x[0], x[1], y[0], y[1]);
            product((ch * kVW + w) * 2 + 1, x[2], x[3], y[2], y[3]);
          } else {
            // eight channels of two keys: the rows' halves side by side, nibble k
            // of both a pair
            const uint32_t x[2] = {__byte_perm(a0, a1, 0x5410), __byte_perm(a0, a1, 0x7632)};
            const uint32_t y[2] = {__byte_perm(a2, a3, 0x5410), __byte_perm(a2, a3, 0x7632)};
            if constexpr (kPg == kI4) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                product((ch * kVW + w) * 4 + 2 * k, int4_pair<true, 0>(x[k]),
                        int4_pair<true, 1>(x[k]), int4_pair<true, 0>(y[k]),
                        int4_pair<true, 1>(y[k]));
                product((ch * kVW + w) * 4 + 2 * k + 1, int4_pair<true, 2>(x[k]),
                        int4_pair<true, 3>(x[k]), int4_pair<true, 2>(y[k]),
                        int4_pair<true, 3>(y[k]));
              }
            } else {
              const uint32_t s0 = e4m3_pair_128(vs[g][0] | vs[g][1] << 8);
              const uint32_t s1 = e4m3_pair_128(vs[g][2] | vs[g][3] << 8);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                product((ch * kVW + w) * 4 + 2 * k, mul_f16x2(e2m1_pair<0>(x[k]), s0),
                        mul_f16x2(e2m1_pair<1>(x[k]), s0), mul_f16x2(e2m1_pair<0>(y[k]), s1),
                        mul_f16x2(e2m1_pair<1>(y[k]), s1));
                product((ch * kVW + w) * 4 + 2 * k + 1, mul_f16x2(e2m1_pair<2>(x[k]), s0),
                        mul_f16x2(e2m1_pair<3>(x[k]), s0), mul_f16x2(e2m1_pair<2>(y[k]), s1),
                        mul_f16x2(e2m1_pair<3>(y[k]), s1));
              }
            }
          }
        }
    if (i + 1 < steps) load_v(cur);
  }

  // the four warps' results, joined in shared memory.  Tile tl of lane (r, c):
  // channels base + 2 tl, + 1 of its chunk, heads 2c, 2c + 1.
  __shared__ float s_acc[kWarps][kRows][kD];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  constexpr int kChunkTiles = Tr::kTiles / Tr::kVChunks;
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[nt][j] += __shfl_xor_sync(~0u, l[nt][j], d);
      const int hd = nt * 8 + 2 * c + j;
      if (r == 0) s_m[warp][hd] = m[nt][j], s_l[warp][hd] = l[nt][j];
#pragma unroll
      for (int ch = 0; ch < Tr::kVChunks; ++ch)
#pragma unroll
        for (int k = 0; k < kChunkTiles; ++k) {
          const int tl = ch * kChunkTiles + k;
          const int d = (ch * 8 + r) * (2 * kChunkTiles) + 2 * k;
          s_acc[warp][hd][d] = acc[nt][tl][j];
          s_acc[warp][hd][d + 1] = acc[nt][tl][j + 2];
        }
    }
  }
  finish_part<TQ, kRows, kD>(p, u, slot, Tr::kUnit, s_acc, s_m, s_l);
  return true;
}

// fp32 pages, which no MMA takes in their precision: the same walk over the
// list, a page's K and V in a warp's registers while the one before is computed,
// with fp32 FMAs.  kD / 4 lanes hold a key's channels, four each, so the scores
// of a key are sums over lanes: kL of them (keys x heads) are summed together,
// each halving of the lanes halving the values too, which takes kL - 1 shuffles
// and leaves lane l the score of head l % kRows.  About 1400 instructions per
// page at 8 heads, 350 cycles of an SM; HBM brings an SM one page in 700.
template <int kD, int kRows>
__device__ __forceinline__ bool attend_part_f32(const SelParams& p, int64_t row, int begin,
                                                int end, int slot) {
  constexpr int kL = kD / 4;           // lanes of a key
  constexpr int kR = 32 / kL;          // keys of one load
  constexpr int kN = kBS / kR;         // loads of a page
  constexpr int kC = kN * kRows / kL;  // scores of a lane
  constexpr int kCN = kN / kC;         // loads of one sum over lanes
  __shared__ __align__(16) float s_acc[kWarps][kRows][kD];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ __align__(16) float s_p[kWarps][kBS][kRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % kL, sub = lane / kL;
  const int first = begin + warp;
  const int steps = end > first ? (end - first + kWarps - 1) / kWarps : 0;
  Listed ahead{0, 0};
  if (first + lane * kWarps < end) ahead = listed(p, row, first + lane * kWarps);
  const Unit u = find_unit(p, row, threadIdx.x == 0);
  if (u.count <= 0) return false;
  const int part = blockIdx.y;
  const int heads = min(p.group - part * kRows, kRows);
  const int head0 = u.h * p.group + part * kRows;
  const int64_t head = (int64_t)u.h * (kBS * kD);
  const int64_t block = (int64_t)p.num_kv_heads * (kBS * kD);
  const float* kbase = static_cast<const float*>(p.k_cache) + head + sub * kD + l * 4;
  const float* vbase = static_cast<const float*>(p.v_cache) + head + sub * kD + l * 4;
  float4 kr[kN], vr[kN];
  // (a skipped entry reads block 0, as over the other types)
  auto load_k = [&](const Entry& e) {
    const float* src = kbase + (int64_t)max(e.phys, 0) * block;
#pragma unroll
    for (int n = 0; n < kN; ++n) kr[n] = __ldg(reinterpret_cast<const float4*>(src + n * kR * kD));
  };
  auto load_v = [&](const Entry& e) {
    const float* src = vbase + (int64_t)max(e.phys, 0) * block;
#pragma unroll
    for (int n = 0; n < kN; ++n) vr[n] = __ldg(reinterpret_cast<const float4*>(src + n * kR * kD));
  };
  Entry held{0, -1};
  auto entry = [&](int i) {
    if ((i & 31) == 0) {
      const int at = first + (i + lane) * kWarps;
      held = Entry{0, -1};
      if (at < end) held = list_entry(p, u, i == 0 ? ahead : listed(p, row, at));
    }
    return Entry{__shfl_sync(~0u, held.block, i & 31), __shfl_sync(~0u, held.phys, i & 31)};
  };
  Entry cur{0, -1};
  if (steps > 0) {
    cur = entry(0);
    load_k(cur);
    load_v(cur);
  }
  float4 q[kRows], acc[kRows];
  const float scale = p.scale * kLog2e;
#pragma unroll
  for (int h = 0; h < kRows; ++h) {
    acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    q[h] = acc[h];
    if (h < heads) {
      q[h] = __ldg(reinterpret_cast<const float4*>(
          static_cast<const float*>(p.q) + (u.t * p.num_q_heads + head0 + h) * kD + l * 4));
      q[h] = make_float4(q[h].x * scale, q[h].y * scale, q[h].z * scale, q[h].w * scale);
    }
  }
  // of head lane % kRows; the sum is that of the lane's own scores
  float m = -INFINITY, sum = 0.f;
  for (int i = 0; i < steps; ++i) {
    float s[kC];
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      float d[kL];
#pragma unroll
      for (int n = 0; n < kCN; ++n) {
        const float4 k = kr[j * kCN + n];
#pragma unroll
        for (int h = 0; h < kRows; ++h)
          d[n * kRows + h] =
              fmaf(k.x, q[h].x, fmaf(k.y, q[h].y, fmaf(k.z, q[h].z, k.w * q[h].w)));
      }
#pragma unroll
      for (int w = kL / 2; w > 0; w >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int x = 0; x < w; ++x) {
          const float give = up ? d[x] : d[x + w];
          const float keep = up ? d[x + w] : d[x];
          d[x] = keep + __shfl_xor_sync(~0u, give, w);
        }
      }
      s[j] = d[0];
    }
    const int keys = cur.phys < 0 ? 0 : min(kBS, u.pos - cur.block * kBS + 1);
    if (i + 1 < steps) {
      cur = entry(i + 1);
      load_k(cur);
    }
    // lane's j-th score: key (j kCN + l / kRows) kR + sub
    if (keys < kBS) {
#pragma unroll
      for (int j = 0; j < kC; ++j)
        if ((j * kCN + l / kRows) * kR + sub >= keys) s[j] = -INFINITY;
#pragma unroll
      for (int n = 0; n < kN; ++n)  // no value that could be NaN
        if (n * kR + sub >= keys) vr[n] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mx = s[0];
#pragma unroll
    for (int j = 1; j < kC; ++j) mx = fmaxf(mx, s[j]);
#pragma unroll
    for (int w = kRows; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, w));
    mx = fmaxf(mx, m);
    if (__any_sync(~0u, mx > m)) {
      const float al = mx == -INFINITY ? 1.f : exp2f(m - mx);
      m = mx;
      sum *= al;
#pragma unroll
      for (int h = 0; h < kRows; ++h) {
        const float f = __shfl_sync(~0u, al, h);
        acc[h] = make_float4(acc[h].x * f, acc[h].y * f, acc[h].z * f, acc[h].w * f);
      }
    }
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const float e = exp2f(s[j] - base);
      sum += e;
      s_p[warp][(j * kCN + l / kRows) * kR + sub][l % kRows] = e;
    }
    __syncwarp();
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const float4 v = vr[n];
#pragma unroll
      for (int h4 = 0; h4 < kRows; h4 += 4) {
        const float4 e = *reinterpret_cast<const float4*>(&s_p[warp][n * kR + sub][h4]);
        const float w[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          float4& a = acc[h4 + h];
          a.x = fmaf(w[h], v.x, a.x);
          a.y = fmaf(w[h], v.y, a.y);
          a.z = fmaf(w[h], v.z, a.z);
          a.w = fmaf(w[h], v.w, a.w);
        }
      }
    }
    __syncwarp();  // the next page's probabilities
    if (i + 1 < steps) load_v(cur);
  }
#pragma unroll
  for (int w = kRows; w < 32; w <<= 1) sum += __shfl_xor_sync(~0u, sum, w);
  if (lane < kRows) s_m[warp][lane] = m, s_l[warp][lane] = sum;
#pragma unroll
  for (int h = 0; h < kRows; ++h) {
    if constexpr (kR == 2) {
      acc[h].x += __shfl_xor_sync(~0u, acc[h].x, 16);
      acc[h].y += __shfl_xor_sync(~0u, acc[h].y, 16);
      acc[h].z += __shfl_xor_sync(~0u, acc[h].z, 16);
      acc[h].w += __shfl_xor_sync(~0u, acc[h].w, 16);
    }
    if (sub == 0) *reinterpret_cast<float4*>(&s_acc[warp][h][l * 4]) = acc[h];
  }
  finish_part<float, kRows, kD>(p, u, slot, 1.f, s_acc, s_m, s_l);
  return true;
}

// The list that begins in this CTA's share and is cut: its parts, place 1 of this
// share and place 0 of the next ones, in order.
template <typename TQ, int kD>
__device__ __forceinline__ void join_cut(const SelParams& p, int2 cut) {
  const int part = blockIdx.y, cta = part * gridDim.x + blockIdx.x;
  const int64_t t = cut.x / p.num_kv_heads;
  const int h = (int)(cut.x - t * p.num_kv_heads);
  const int heads = min(p.group - part * p.head_rows, p.head_rows);
  const int parts = cut.y;
  auto place = [&](int k) {
    return (2 * (int64_t)(cta + k) + (k == 0 ? 1 : 0)) * p.head_rows;
  };
  // Four channels per thread; the parts' loads go out together, eight at a time:
  // one token's lists of 17 parts 9.3 us, with four at a time 10.1, with sixteen
  // 9.1, but the batch of 64 tokens 92 instead of 89.
  constexpr int kQuads = kD / 4, kBatch = 8;
  for (int i = threadIdx.x; i < heads * kQuads; i += kJoinThreads) {
    const int hd = i / kQuads, d = (i - hd * kQuads) * 4;
    float mx = -INFINITY, ls = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < parts; k0 += kBatch) {
      float2 ml[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int64_t at = place(min(k0 + j, parts - 1)) + hd;
        ml[j] = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
        v[j] = *reinterpret_cast<const float4*>(p.part + at * kD + d);
      }
      // a place past the last part holds that one again: nothing of it, not even 0
      // times its sum, which may be infinite.  (Selected here: with a branch below
      // the loads go out one by one, and one token takes 12.2 us.)
#pragma unroll
      for (int j = 1; j < kBatch; ++j)
        if (k0 + j >= parts) {
          ml[j] = make_float2(-INFINITY, 0.f);
          v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      float top = mx;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) top = fmaxf(top, ml[j].x);
      const float old = mx == -INFINITY ? 0.f : exp2f(mx - top);
      ls *= old;
      a = make_float4(a.x * old, a.y * old, a.z * old, a.w * old);
      mx = top;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const float f = ml[j].x == -INFINITY ? 0.f : exp2f(ml[j].x - top);
        ls = fmaf(f, ml[j].y, ls);
        a.x = fmaf(f, v[j].x, a.x);
        a.y = fmaf(f, v[j].y, a.y);
        a.z = fmaf(f, v[j].z, a.z);
        a.w = fmaf(f, v[j].w, a.w);
      }
    }
    TQ* out = static_cast<TQ*>(p.out) +
              (t * p.num_q_heads + h * p.group + part * p.head_rows + hd) * kD + d;
    const float o[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = from_f32<TQ>(ls == 0.f ? 0.f : o[e] / ls * p.v_scale);
  }
}

// Behind the shares: CTA i joins the list that begins in share i and is cut
// (the part there, then the first part of each share it goes on through), and
// writes the zeros of the rows i, i + gridDim.x, .. whose list is empty: a
// thread looks at a row's count, its warp then writes the empty ones.
template <typename TQ, int kD>
__global__ void __launch_bounds__(kJoinThreads) selected_join_kernel(const SelParams p) {
  const int part = blockIdx.y, lane = threadIdx.x & 31;
  const int64_t rows = p.s.num_tokens * p.num_kv_heads, step = gridDim.x;
  auto empty = [&](int64_t row) { return row < rows && list_length(p, row) == 0; };
  // These CTAs start as the shares' end: what can be read before goes out first,
  // and the zeros come last (before the join: one token's 8 lists 12.0 us, not 10.5).
  const bool here = empty(blockIdx.x + threadIdx.x * step);
  if (part == 0)
    check_requests(p.s, (int64_t)blockIdx.x * kJoinThreads + threadIdx.x,
                   step * kJoinThreads);
  pdl_wait();  // the shares' results
  const int2 cut = p.cut[part * gridDim.x + blockIdx.x];
  if (cut.x >= 0) join_cut<TQ, kD>(p, cut);
  for (int64_t first = 0; blockIdx.x + first * step < rows; first += kJoinThreads) {
    const int64_t mine = first + threadIdx.x;
    unsigned todo = __ballot_sync(~0u, first == 0 ? here : empty(blockIdx.x + mine * step));
    for (; todo != 0; todo &= todo - 1) {
      const int64_t row = blockIdx.x + (mine - lane + __ffs(todo) - 1) * step;
      const Unit u = find_unit(p, row, part == 0 && lane == 0);
      if (u.count < 0) continue;
      const int heads = min(p.group - part * p.head_rows, p.head_rows);
      TQ* out = static_cast<TQ*>(p.out) +
                (u.t * p.num_q_heads + u.h * p.group + part * p.head_rows) * kD;
      for (int i = lane; i < heads * kD; i += 32) out[i] = from_f32<TQ>(0.f);
    }
  }
}

cudaError_t launched() {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename TQ, int kPg, int kD>
cudaError_t launch_d(const SelParams& p, const SelectedPlan& plan, cudaStream_t stream) {
  const dim3 grid((unsigned)plan.shares, (unsigned)plan.head_parts);
  constexpr int kRows = kPg == kF32 ? 4 : 8;  // or twice as many
  if (p.head_rows == kRows)
    selected_kernel<TQ, kPg, kD, kRows><<<grid, kThreads, 0, stream>>>(p);
  else
    selected_kernel<TQ, kPg, kD, 2 * kRows><<<grid, kThreads, 0, stream>>>(p);
  cudaError_t e = launched();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, selected_join_kernel<TQ, kD>, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename TQ, int kPg>
cudaError_t launch_t(const SelParams& p, int head_dim, const SelectedPlan& plan,
                       cudaStream_t stream) {
  return head_dim == 128 ? launch_d<TQ, kPg, 128>(p, plan, stream)
                         : launch_d<TQ, kPg, 64>(p, plan, stream);
}

}  // namespace

namespace {

SelectedPlan plan_for(bool fp32, int64_t num_tokens, int num_q_heads, int num_kv_heads,
                      int head_dim, int max_selected, int num_sms) {
  SelectedPlan pl{};
  const int group = num_q_heads / num_kv_heads;
  pl.head_rows = fp32 ? (group <= 4 ? 4 : 8) : (group <= 8 ? 8 : 16);
  pl.head_parts = (group + pl.head_rows - 1) / pl.head_rows;
  // a share per resident CTA, fewer where the shares would be below kMinShare
  const int64_t units = num_tokens * num_kv_heads * ((int64_t)max_selected + kRowCost);
  const int64_t slots = (int64_t)ctas_per_sm(fp32, pl.head_rows) * num_sms;
  pl.shares = std::min(std::max<int64_t>(1, slots / pl.head_parts),
                       (units + kMinShare - 1) / kMinShare);
  const int64_t parts = 2 * pl.shares * pl.head_parts * pl.head_rows;
  pl.off_ml = parts * head_dim * (int64_t)sizeof(float);
  pl.off_cut = pl.off_ml + parts * 2 * (int64_t)sizeof(float);
  pl.bytes = pl.off_cut + pl.shares * pl.head_parts * (int64_t)sizeof(int2);
  return pl;
}

}  // namespace

SelectedPlan make_selected_plan(pa_dtype cache_dtype, int64_t num_tokens, int num_q_heads,
                                int num_kv_heads, int head_dim, int max_selected,
                                int num_sms) {
  const SelectedPlan a = plan_for(false, num_tokens, num_q_heads, num_kv_heads, head_dim,
                                  max_selected, num_sms);
  const SelectedPlan b =
      plan_for(true, num_tokens, num_q_heads, num_kv_heads, head_dim, max_selected, num_sms);
  SelectedPlan pl = cache_dtype == PA_F32 ? b : a;
  pl.bytes = std::max(a.bytes, b.bytes);  // one size for caches of every type
  return pl;
}

cudaError_t launch_attention_selected(const StepView& s, const SelectedPlan& plan,
                                      const SelectedArgs& a, cudaStream_t stream) {
  SelParams p{};
  p.s = s;
  p.q = a.q;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.head_rows = plan.head_rows;
  p.selected = a.selected;
  p.num_selected = a.num_selected;
  p.max_selected = a.max_selected;
  p.scale = a.scale;
  const bool scaled = a.cache_dtype == PA_FP8_E4M3 || a.cache_dtype == PA_NVFP4;
  p.k_scale = scaled ? a.k_scale : 1.0f;
  p.v_scale = scaled ? a.v_scale : 1.0f;
  p.out = a.out;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.part = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + plan.off_ml);
  p.cut = reinterpret_cast<int2*>(ws + plan.off_cut);
  const bool bf = a.q_dtype == PA_BF16;
  switch (a.cache_dtype) {
    case PA_F32: return launch_t<float, kF32>(p, a.head_dim, plan, stream);
    case PA_F16: return launch_t<__half, kH16>(p, a.head_dim, plan, stream);
    case PA_BF16: return launch_t<__nv_bfloat16, kB16>(p, a.head_dim, plan, stream);
    case PA_FP8_E4M3:
      return bf ? launch_t<__nv_bfloat16, kF8>(p, a.head_dim, plan, stream)
                : launch_t<__half, kF8>(p, a.head_dim, plan, stream);
    case PA_INT4:
      return bf ? launch_t<__nv_bfloat16, kI4>(p, a.head_dim, plan, stream)
                : launch_t<__half, kI4>(p, a.head_dim, plan, stream);
    case PA_NVFP4:
      return bf ? launch_t<__nv_bfloat16, kN4>(p, a.head_dim, plan, stream)
                : launch_t<__half, kN4>(p, a.head_dim, plan, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pa
