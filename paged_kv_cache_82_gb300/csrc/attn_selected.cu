// attn_selected.cu -- attention of each token over a list of its cache blocks
// (pa_attention_selected).
//
//   out = sum_j softmax(scale <q, k_j>)_j v_j  over the keys j of the listed
//   blocks up to the token's own position; a list of no blocks gives zeros.
//
// A row is one (token, KV head) with its list; all rows' list entries in a row,
// end to end, are cut into equal shares, one CTA each, as many as are resident
// (every CTA sums the rows' list lengths for itself).  A share holds whole
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
#include <algorithm>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kJoinThreads = 256;  // 8 heads x 128 channels, four per thread
#ifndef PA_SEL_SHARE
#define PA_SEL_SHARE 8
#endif
constexpr int kMinShare = PA_SEL_SHARE;  // list entries of a CTA, at least
constexpr float kLog2e = 1.4426950408889634f;

enum : int { kB16 = 0, kH16 = 1, kF8 = 2 };  // bf16, f16, E4M3 pages

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
  // parts of lists, two per CTA: its first and its last (see write_part)
  float* part;     // [CTA][2][head_rows][D]
  float* part_ml;  // [CTA][2][head_rows][2]: m, l
  int2* cut;       // [CTA]: the row whose list begins here and is cut (-1: none)
};

// A row: its token, request, position and list length (-1: the token belongs
// to no request, or its metadata is broken).
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
  if (!q.in) {
    u.count = -1;
  } else if (!q.m.ok) {
    if (tell) flag_error(p.s.err, PA_DEV_ERR_METADATA);
    u.count = -1;
  } else if (u.count < 0 || u.count > p.max_selected) {
    if (tell) flag_error(p.s.err, PA_DEV_ERR_METADATA);
    u.count = 0;
  }
  return u;
}

// Entry i of the unit's list: the logical block and its physical block (-1:
// skipped, with a flag -- not above the entry before it, past the token's
// position, or a bad physical id).
struct Entry {
  int block, phys;
};
__device__ __forceinline__ Entry list_entry(const SelParams& p, const Unit& u, int i) {
  const int32_t* list =
      p.selected + (u.t * p.num_kv_heads + u.h) * p.max_selected;
  Entry e;
  e.block = __ldg(list + i);
  const int before = i > 0 ? __ldg(list + i - 1) : -1;
  e.phys = -1;
  if (e.block <= before || e.block < 0 || e.block > u.pos / kBS) {
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

// ---------------------------------------------------------------------------
// the types without an MMA form (fp32, 4-bit pages): one warp per (token,
// query head)'s share of the list, four warps to a list
// ---------------------------------------------------------------------------
struct F32Page {};
struct Int4Page {};
struct Nvfp4Page {};

template <typename TP, int kD>
__device__ __forceinline__ float page_elem(const void* base, int64_t page, int o, int d) {
  if constexpr (std::is_same<TP, F32Page>::value) {
    return __ldg(static_cast<const float*>(base) + (page * kBS + o) * kD + d);
  } else {
    constexpr bool nv = std::is_same<TP, Nvfp4Page>::value;
    const uint8_t* pg =
        static_cast<const uint8_t*>(base) + page * (nv ? 9 * kD : 8 * kD + 64);
    const uint32_t byte = __ldg(pg + o * (kD / 2) + d / 2);
    const uint32_t nib = (d & 1) ? byte >> 4 : byte & 15u;
    if constexpr (nv)
      return e4m3_to_f32(__ldg(pg + kBS * (kD / 2) + o * (kD / 16) + d / 16)) *
             e2m1_to_f32(nib);
    else
      return __ldg(reinterpret_cast<const float*>(pg + kBS * (kD / 2) + 4 * o)) *
             (float)((int)(nib ^ 8u) - 8);
  }
}

template <typename TQ, typename TP, int kD>
__global__ void __launch_bounds__(kThreads) selected_generic_kernel(const SelParams p) {
  constexpr int kPer = kD / 32;
  __shared__ float s_acc[kWarps][kD], s_m[kWarps], s_l[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x / p.num_q_heads;
  const int hq = (int)(blockIdx.x % p.num_q_heads);
  const Unit u = find_unit(p, t * p.num_kv_heads + hq / p.group, threadIdx.x == 0);
  if (u.count < 0) return;
  const TQ* qp = static_cast<const TQ*>(p.q) + (t * p.num_q_heads + hq) * kD;
  float qv[kPer], acc[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    qv[k] = to_f32(qp[lane + 32 * k]) * p.scale * p.k_scale;
    acc[k] = 0.f;
  }
  for (int i = warp; i < u.count; i += kWarps) {
    const Entry e = list_entry(p, u, i);
    if (e.phys < 0) continue;
    const int64_t page = (int64_t)e.phys * p.num_kv_heads + u.h;
    const int keys = min(kBS, u.pos - e.block * kBS + 1);
    for (int o = 0; o < keys; ++o) {
      float dot = 0.f;
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        dot += qv[k] * page_elem<TP, kD>(p.k_cache, page, o, lane + 32 * k);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(~0u, dot, d);
      const float mn = fmaxf(m, dot);
      if (mn == -INFINITY) continue;  // nothing but -inf so far
      const float al = expf(m - mn), pj = expf(dot - mn);
      l = l * al + pj;
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        acc[k] = acc[k] * al + pj * page_elem<TP, kD>(p.v_cache, page, o, lane + 32 * k);
      m = mn;
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) s_acc[warp][lane + 32 * k] = acc[k];
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
  __syncthreads();
  float mx = -INFINITY;
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w]);
  for (int d = threadIdx.x; d < kD; d += kThreads) {
    float a = 0.f, ls = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float f = s_m[w] == -INFINITY ? 0.f : expf(s_m[w] - mx);
      a += f * s_acc[w][d];
      ls += f * s_l[w];
    }
    static_cast<TQ*>(p.out)[(t * p.num_q_heads + hq) * kD + d] =
        from_f32<TQ>(ls > 0.f ? a / ls * p.v_scale : ls);
  }
}

// ---------------------------------------------------------------------------
// the MMA form
// ---------------------------------------------------------------------------
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


// A lane's words of one row of a page: 16 bytes per chunk
template <int kPg, int kD>
struct PageTraits {
  static constexpr int kEB = kPg == kF8 ? 1 : 2;
  static constexpr int kRowBytes = kD * kEB;
  // K: lane (r, c) reads 16 bytes at 16 c + 64 i of rows r and r + 8
  static constexpr int kKChunks = kRowBytes / 64;
  // V: lane (r, c) reads kVBytes at kVBytes r (+ 8 kVBytes i) of the rows
  // 2c, 2c + 1, 2c + 8, 2c + 9
  static constexpr int kVBytes = kRowBytes >= 128 ? 16 : 8;
  static constexpr int kVChunks = kRowBytes / (8 * kVBytes);
  static constexpr int kTiles = kD / 16;  // m16 tiles of the output's channels
  // Pages of one step: 8 KB of K and V in a warp's registers, whatever the
  // type, are on their way while the step before is computed (one page of
  // 8-bit types leaves half the bytes in flight: 57 instead of PLACEHOLDER us for 32 tokens'
  // 256 blocks of 8 KV heads).
  static constexpr int kPages = 4096 / (kBS * kRowBytes);
};

// CTAs per SM that the kernels are built for: what the accumulators of 8 (kNT
// = 1) or 16 query heads leave of the registers
constexpr int ctas_per_sm(int head_rows) { return head_rows == 8 ? 3 : 2; }

// Entries of a row's list that count: none of a row past the last request.
__device__ __forceinline__ int list_length(const SelParams& p, int64_t row) {
  const int c = __ldg(p.num_selected + row);
  return c > 0 && c <= p.max_selected ? c : 0;
}

// A CTA's share of all the rows' list entries.
struct Share {
  int64_t begin, end;  // entries
  int64_t size;        // of every share
  int64_t row;         // the row that `begin` lies in,
  int64_t row_begin;   // and where its list begins
};

__device__ __forceinline__ int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

// Every thread sums a contiguous part of the rows; the one whose part holds
// the share's first entry walks it.
__device__ __forceinline__ Share find_share(const SelParams& p, int64_t rows) {
  __shared__ int64_t warp_sums[32], total, s_row, s_row_begin;
  const int64_t part = (rows + kThreads - 1) / kThreads;
  const int64_t lo = least(rows, threadIdx.x * part), hi = least(rows, lo + part);
  int64_t sum = 0;
  for (int64_t i = lo; i < hi; ++i) sum += list_length(p, i);
  const int64_t before = block_scan_excl(sum, &total, warp_sums);
  Share s;
  s.size = (total + gridDim.x - 1) / gridDim.x;
  if (s.size < kMinShare) s.size = kMinShare;
  s.begin = least(total, blockIdx.x * s.size);
  s.end = least(total, s.begin + s.size);
  if (s.begin < s.end && s.begin >= before && s.begin < before + sum) {
    int64_t at = before, i = lo;
    for (int c; at + (c = list_length(p, i)) <= s.begin; ++i) at += c;
    s_row = i;
    s_row_begin = at;
  }
  __syncthreads();
  s.row = s_row;
  s.row_begin = s_row_begin;
  return s;
}

template <typename TQ, int kPg, int kD, int kNT>
__device__ __forceinline__ void attend_part(const SelParams& p, const Unit& u, int begin,
                                            int end, int slot);

template <typename TQ, int kPg, int kD, int kNT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(8 * kNT))
selected_kernel(const SelParams p) {
  pdl_launch_dependents();
  // rows of tokens up to the last request's
  const int64_t last = __ldg(p.s.query_start_loc + p.s.num_seqs);
  const int64_t tokens = last < 0 ? 0 : least(last, p.s.num_tokens);
  const int64_t rows = tokens * p.num_kv_heads;
  const Share sh = find_share(p, rows);
  const int cta = blockIdx.y * gridDim.x + blockIdx.x;
  int2 cut = make_int2(-1, 0);
  int64_t at = sh.begin, row = sh.row, row_begin = sh.row_begin;
  while (at < sh.end) {
    const int64_t row_end = row_begin + list_length(p, row);
    if (row_end > at) {
      const int64_t end = least(row_end, sh.end);
      const Unit u = find_unit(p, row, threadIdx.x == 0);
      // -1: the whole list is here; else the CTA's place for a part: 0 for its
      // first entry's row, 1 for the row that goes on in the next CTA
      const int slot = at == row_begin && end == row_end ? -1 : at == sh.begin ? 0 : 1;
      if (u.count > 0) {
        attend_part<TQ, kPg, kD, kNT>(p, u, (int)(at - row_begin), (int)(end - row_begin),
                                      slot);
        if (at == row_begin && end < row_end)
          // parts x 2 + the place of the first
          cut = make_int2((int)row,
                          (int)((row_end - 1) / sh.size - blockIdx.x + 1) * 2 + slot);
      }
      at = end;
    }
    row_begin = row_end;
    ++row;
  }
  if (threadIdx.x == 0) p.cut[cta] = cut;
}

// Entries begin .. end - 1 of a row's list: to the output if that is all of it
// (slot < 0), else to the CTA's place for a part.
template <typename TQ, int kPg, int kD, int kNT>
__device__ __forceinline__ void attend_part(const SelParams& p, const Unit& u, int begin,
                                            int end, int slot) {
  using Tr = PageTraits<kPg, kD>;
  constexpr bool kBF = kPg == kB16;
  constexpr int kRows = 8 * kNT;  // query heads, at most
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, c = lane & 3;
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

  constexpr int kP = Tr::kPages;
  uint4 kr[kP][2][Tr::kKChunks];
  uint32_t vr[kP][4][Tr::kVChunks][Tr::kVBytes / 4];
  constexpr int64_t kPageBytes = kBS * (int64_t)Tr::kRowBytes;
  const uint8_t* kbase = static_cast<const uint8_t*>(p.k_cache) + (int64_t)u.h * kPageBytes;
  const uint8_t* vbase = static_cast<const uint8_t*>(p.v_cache) + (int64_t)u.h * kPageBytes;
  const int64_t block_bytes = kPageBytes * p.num_kv_heads;
  const int koff = r * Tr::kRowBytes + c * 16;

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
      const uint8_t* src = kbase + (int64_t)max(en[g].phys, 0) * block_bytes + koff;
#pragma unroll
      for (int i = 0; i < Tr::kKChunks; ++i) {
        kr[g][0][i] = __ldg(reinterpret_cast<const uint4*>(src + 64 * i));
        kr[g][1][i] = __ldg(reinterpret_cast<const uint4*>(src + 8 * Tr::kRowBytes + 64 * i));
      }
    }
  };
  auto load_v = [&](const Entry (&en)[kP]) {
#pragma unroll
    for (int g = 0; g < kP; ++g) {
      const uint8_t* src = vbase + (int64_t)max(en[g].phys, 0) * block_bytes +
                           2 * c * Tr::kRowBytes + r * Tr::kVBytes;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int i = 0; i < Tr::kVChunks; ++i) {
          const uint8_t* at =
              src + ((j & 1) + 8 * (j >> 1)) * Tr::kRowBytes + i * 8 * Tr::kVBytes;
          if constexpr (Tr::kVBytes == 16) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(at));
            vr[g][j][i][0] = v.x; vr[g][j][i][1] = v.y;
            vr[g][j][i][2] = v.z; vr[g][j][i][3] = v.w;
          } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
            vr[g][j][i][0] = v.x; vr[g][j][i][1] = v.y;
          }
        }
      }
    }
  };

  // The warp's steps: kP entries in a row from begin + kP warp, then kP kWarps
  // further on.  The lanes hold the next 32 of the warp's entries.
  const int first = begin + kP * warp;
  const int steps = end > first ? (end - first + kP * kWarps - 1) / (kP * kWarps) : 0;
  Entry held{0, -1};
  auto entries = [&](int step, Entry (&en)[kP]) {
    const int i = step * kP;  // of the warp's entries
    if ((i & 31) == 0) {
      const int mine = i + lane;
      const int at = first + (mine / kP) * (kP * kWarps) + mine % kP;
      held = Entry{0, -1};
      if (at < end) held = list_entry(p, u, at);
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

  // Q operand words, in the channel order of the lane's K words.  Over FP8
  // pages the products are in f16: a power of two brings the unit's largest
  // query into f16's range, and leaves through the score's scale.
  uint32_t qw[kNT][Tr::kKChunks][kPg == kF8 ? 8 : 4];
  float score_scale = p.scale * p.k_scale * kLog2e;
  {
    constexpr int kE = 16 / Tr::kEB;  // channels of one chunk
    float x[kNT][Tr::kKChunks][kE];
    float big = 0.f;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int i = 0; i < Tr::kKChunks; ++i) {
        const int hd = nt * 8 + r;
        const TQ* src = static_cast<const TQ*>(p.q) +
                        (u.t * p.num_q_heads + head0 + hd) * kD + (c + 4 * i) * kE;
        uint4 w[kE / 8];
#pragma unroll
        for (int e = 0; e < kE / 8; ++e)
          w[e] = hd < heads ? __ldg(reinterpret_cast<const uint4*>(src) + e)
                            : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          x[nt][i][e] = to_f32(reinterpret_cast<const TQ*>(w)[e]);
          big = fmaxf(big, fabsf(x[nt][i][e]));
        }
      }
    // a scale of either sign, or 0: the score's stays positive
    float down = score_scale > 0.f ? 1.f : score_scale < 0.f ? -1.f : 0.f;
    score_scale = score_scale == 0.f ? 1.f : fabsf(score_scale);
    if constexpr (kPg == kF8) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, d));
      if (big > 16384.f && big < INFINITY) {
        const int ex = ilogbf(big) - 13;
        down *= exp2f((float)-ex);
        score_scale *= exp2f((float)ex);
      }
    }
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int i = 0; i < Tr::kKChunks; ++i)
#pragma unroll
        for (int w = 0; w < kE / 2; ++w)
          qw[nt][i][w] = pack2<kBF>(x[nt][i][2 * w] * down, x[nt][i][2 * w + 1] * down);
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
        const uint32_t w0[4] = {kr[g][0][ch].x, kr[g][0][ch].y, kr[g][0][ch].z, kr[g][0][ch].w};
        const uint32_t w1[4] = {kr[g][1][ch].x, kr[g][1][ch].y, kr[g][1][ch].z, kr[g][1][ch].w};
        if constexpr (kPg == kF8) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a[4];
            e4m3x4_to_f16x2x2(w0[w], a[0], a[2]);
            e4m3x4_to_f16x2x2(w1[w], a[1], a[3]);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
              mma16816<false>(s[g][nt], a, qw[nt][ch][2 * w], qw[nt][ch][2 * w + 1]);
          }
        } else {
#pragma unroll
          for (int w = 0; w < 4; w += 2) {
            const uint32_t a[4] = {w0[w], w1[w], w0[w + 1], w1[w + 1]};
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
              mma16816<kBF>(s[g][nt], a, qw[nt][ch][w], qw[nt][ch][w + 1]);
          }
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
              for (int w = 0; w < Tr::kVBytes / 4; ++w) vr[g][j][ch][w] = 0;
      }
    }
    // softmax over the step's keys; m: the largest score times score_scale (> 0)
    uint32_t pb[kP][kNT][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      float mx[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mx[j] = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
#pragma unroll
        for (int g = 1; g < kP; ++g) mx[j] = fmaxf(mx[j], fmaxf(s[g][nt][j], s[g][nt][j + 2]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) mx[j] = fmaxf(mx[j], __shfl_xor_sync(~0u, mx[j], d));
        mx[j] = fmaxf(mx[j] * score_scale, m[nt][j]);
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
        const float p0 = exp2_fast(fmaf(s[g][nt][0], score_scale, m0));
        const float p1 = exp2_fast(fmaf(s[g][nt][1], score_scale, m1));
        const float p2 = exp2_fast(fmaf(s[g][nt][2], score_scale, m0));
        const float p3 = exp2_fast(fmaf(s[g][nt][3], score_scale, m1));
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        // keys as rows -> heads as rows: the second product's operand
        pb[g][nt][0] = transpose8x8(pack2<kBF>(p0, p1));
        pb[g][nt][1] = transpose8x8(pack2<kBF>(p2, p3));
      }
    }
    // O^T += V^T P^T: channels as rows
#pragma unroll
    for (int g = 0; g < kP; ++g)
#pragma unroll
      for (int ch = 0; ch < Tr::kVChunks; ++ch)
#pragma unroll
        for (int w = 0; w < Tr::kVBytes / 4; ++w) {
          const uint32_t a0 = vr[g][0][ch][w], a1 = vr[g][1][ch][w];
          const uint32_t a2 = vr[g][2][ch][w], a3 = vr[g][3][ch][w];
          if constexpr (kPg == kF8) {
            // four channels of two keys: bytes of the two rows side by side
            const uint32_t l01 = __byte_perm(a0, a1, 0x5140), h01 = __byte_perm(a0, a1, 0x7362);
            const uint32_t l23 = __byte_perm(a2, a3, 0x5140), h23 = __byte_perm(a2, a3, 0x7362);
            uint32_t x[4], y[4];
            e4m3x4_to_f16x2x2(l01, x[0], x[1]);
            e4m3x4_to_f16x2x2(h01, x[2], x[3]);
            e4m3x4_to_f16x2x2(l23, y[0], y[1]);
            e4m3x4_to_f16x2x2(h23, y[2], y[3]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a[4] = {x[2 * k], x[2 * k + 1], y[2 * k], y[2 * k + 1]};
#pragma unroll
              for (int nt = 0; nt < kNT; ++nt)
                mma16816<false>(acc[nt][(ch * (Tr::kVBytes / 4) + w) * 2 + k], a,
                                pb[g][nt][0], pb[g][nt][1]);
            }
          } else {
            const uint32_t a[4] = {__byte_perm(a0, a1, 0x5410), __byte_perm(a0, a1, 0x7632),
                                   __byte_perm(a2, a3, 0x5410), __byte_perm(a2, a3, 0x7632)};
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
              mma16816<kBF>(acc[nt][ch * (Tr::kVBytes / 4) + w], a, pb[g][nt][0], pb[g][nt][1]);
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

// Behind the shares: CTA i joins the list that begins in share i and is cut
// (the part there, then the first part of each share it goes on through), and
// writes the zeros of the rows i, i + gridDim.x, .. whose list is empty.
template <typename TQ, int kD>
__global__ void __launch_bounds__(kJoinThreads) selected_join_kernel(const SelParams p) {
  const int part = blockIdx.y;
  const int64_t rows = p.s.num_tokens * p.num_kv_heads;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    if (list_length(p, row) > 0) continue;
    const Unit u = find_unit(p, row, part == 0 && threadIdx.x == 0);
    if (u.count < 0) continue;
    const int heads = min(p.group - part * p.head_rows, p.head_rows);
    TQ* out = static_cast<TQ*>(p.out) +
              (u.t * p.num_q_heads + u.h * p.group + part * p.head_rows) * kD;
    for (int i = threadIdx.x; i < heads * kD; i += kJoinThreads) out[i] = from_f32<TQ>(0.f);
  }
  pdl_wait();  // the shares' results
  const int cta = part * gridDim.x + blockIdx.x;
  const int2 cut = p.cut[cta];
  if (cut.x < 0) return;
  const int64_t t = cut.x / p.num_kv_heads;
  const int h = (int)(cut.x - t * p.num_kv_heads);
  const int heads = min(p.group - part * p.head_rows, p.head_rows);
  // the list's parts: place 0 or 1 of this share, place 0 of the next ones
  const int parts = cut.y / 2;
  auto place = [&](int k) {
    return (2 * (int64_t)(cta + k) + (k == 0 ? cut.y % 2 : 0)) * p.head_rows;
  };
  // four channels per thread; the parts' loads go out together, four at a time
  constexpr int kQuads = kD / 4, kBatch = 4;
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
      float top = mx;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) top = fmaxf(top, ml[j].x);
      const float old = mx == -INFINITY ? 0.f : exp2f(mx - top);
      ls *= old;
      a = make_float4(a.x * old, a.y * old, a.z * old, a.w * old);
      mx = top;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const float f =
            k0 + j >= parts || ml[j].x == -INFINITY ? 0.f : exp2f(ml[j].x - top);
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

cudaError_t launched() {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename TQ, typename TP>
cudaError_t launch_generic(const SelParams& p, int head_dim, cudaStream_t stream) {
  const int64_t grid = p.s.num_tokens * p.num_q_heads;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  if (head_dim == 128)
    selected_generic_kernel<TQ, TP, 128><<<(unsigned)grid, kThreads, 0, stream>>>(p);
  else
    selected_generic_kernel<TQ, TP, 64><<<(unsigned)grid, kThreads, 0, stream>>>(p);
  return launched();
}

template <typename TQ, int kPg, int kD>
cudaError_t launch_mma_d(const SelParams& p, const SelectedPlan& plan, cudaStream_t stream) {
  const dim3 grid((unsigned)plan.shares, (unsigned)plan.head_parts);
  if (p.head_rows == 8)
    selected_kernel<TQ, kPg, kD, 1><<<grid, kThreads, 0, stream>>>(p);
  else
    selected_kernel<TQ, kPg, kD, 2><<<grid, kThreads, 0, stream>>>(p);
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
cudaError_t launch_mma(const SelParams& p, int head_dim, const SelectedPlan& plan,
                       cudaStream_t stream) {
  return head_dim == 128 ? launch_mma_d<TQ, kPg, 128>(p, plan, stream)
                         : launch_mma_d<TQ, kPg, 64>(p, plan, stream);
}

}  // namespace

SelectedPlan make_selected_plan(int64_t num_tokens, int num_q_heads, int num_kv_heads,
                                int head_dim, int max_selected, int num_sms) {
  SelectedPlan pl{};
  const int group = num_q_heads / num_kv_heads;
  pl.head_rows = group <= 8 ? 8 : 16;
  pl.head_parts = (group + pl.head_rows - 1) / pl.head_rows;
  // a share per resident CTA, fewer where shares would be below kMinShare
  const int64_t entries = num_tokens * num_kv_heads * (int64_t)max_selected;
  const int64_t slots = (int64_t)ctas_per_sm(pl.head_rows) * num_sms;
  pl.shares = std::min(std::max<int64_t>(1, slots / pl.head_parts),
                       (entries + kMinShare - 1) / kMinShare);
  const int64_t parts = 2 * pl.shares * pl.head_parts * pl.head_rows;
  pl.off_ml = parts * head_dim * (int64_t)sizeof(float);
  pl.off_cut = pl.off_ml + parts * 2 * (int64_t)sizeof(float);
  pl.bytes = pl.off_cut + pl.shares * pl.head_parts * (int64_t)sizeof(int2);
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
    case PA_F32: return launch_generic<float, F32Page>(p, a.head_dim, stream);
    case PA_F16: return launch_mma<__half, kH16>(p, a.head_dim, plan, stream);
    case PA_BF16:
      return launch_mma<__nv_bfloat16, kB16>(p, a.head_dim, plan, stream);
    case PA_FP8_E4M3:
      return bf ? launch_mma<__nv_bfloat16, kF8>(p, a.head_dim, plan, stream)
                : launch_mma<__half, kF8>(p, a.head_dim, plan, stream);
    case PA_INT4:
      return bf ? launch_generic<__nv_bfloat16, Int4Page>(p, a.head_dim, stream)
                : launch_generic<__half, Int4Page>(p, a.head_dim, stream);
    case PA_NVFP4:
      return bf ? launch_generic<__nv_bfloat16, Nvfp4Page>(p, a.head_dim, stream)
                : launch_generic<__half, Nvfp4Page>(p, a.head_dim, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pa
