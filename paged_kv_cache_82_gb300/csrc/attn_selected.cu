// attn_selected.cu -- attention of each token over a list of its cache blocks
// (pa_attention_selected).
//
//   out = sum_j softmax(scale <q, k_j>)_j v_j  over the keys j of the listed
//   blocks up to the token's own position; a list of no blocks gives zeros.
//
// A work unit is one (token, KV head, up to 16 of its query heads); its list
// is cut into `splits` ranges when there are few units, and a second kernel
// joins the ranges' partial results in order.
//
// The unit reads each listed block's K and V page once and does 4 G multiply-
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

#include <cooperative_groups.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kWarps = 4;
#ifndef PA_SEL_AHEAD
#define PA_SEL_AHEAD 2
#endif
constexpr int kAhead = PA_SEL_AHEAD;  // pages asked into L2 before their loads
constexpr int kThreads = kWarps * 32;
#ifndef PA_SEL_WAVES
#define PA_SEL_WAVES 2
#endif
constexpr int kSelWaves = PA_SEL_WAVES;
constexpr float kLog2e = 1.4426950408889634f;

enum : int { kB16 = 0, kH16 = 1, kF8 = 2 };  // bf16, f16, E4M3 pages

struct SelParams {
  StepView s;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  int num_q_heads, num_kv_heads, group;
  int head_parts, cluster, splits;  // ranges of a list: cluster x splits
  const int32_t* selected;
  const int32_t* num_selected;
  int max_selected;
  float scale, k_scale, v_scale;
  void* out;
  float* part;     // [unit][split][head_rows][D]
  float* part_ml;  // [unit][split][head_rows][2]: m, l
  int head_rows;
};

// Token t of a unit: its request, position and list length (-1: the token
// belongs to no request, or its metadata is broken).
struct Unit {
  int64_t t;
  int h, part;  // KV head, part of its group
  int r, pos, count;
};

__device__ __forceinline__ Unit find_unit(const SelParams& p, int64_t unit, bool tell) {
  Unit u;
  u.part = (int)(unit % p.head_parts);
  const int64_t th = unit / p.head_parts;
  u.h = (int)(th % p.num_kv_heads);
  u.t = th / p.num_kv_heads;
  u.count = __ldg(p.num_selected + u.t * p.num_kv_heads + u.h);
  u.r = warp_find_request(p.s.query_start_loc, p.s.num_seqs, u.t);
  const ReqMeta m =
      load_req(p.s.query_start_loc, p.s.seq_lens, u.r, p.s.num_tokens,
               p.s.max_query_len, p.s.max_seq_len, p.s.max_blocks_per_seq);
  u.pos = m.L - m.n + (int)(u.t - m.q0);
  if (u.t < m.q0 || u.t >= (int64_t)m.q0 + m.n) {
    u.count = -1;
  } else if (!m.ok) {
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
  Unit u = find_unit(p, (t * p.num_kv_heads + hq / p.group) * p.head_parts,
                     threadIdx.x == 0);
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
};

template <typename TQ, int kPg, int kD, int kNT>
__global__ void __launch_bounds__(kThreads)
selected_kernel(const SelParams p) {
  using Tr = PageTraits<kPg, kD>;
  constexpr bool kBF = kPg == kB16;
  constexpr int kRows = 8 * kNT;  // query heads of the unit, at most
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, c = lane & 3;
  // CTA (unit, split, rank): the ranks of one (unit, split) are a cluster
  const int ranges = p.cluster * p.splits;
  const int64_t unit = blockIdx.x / ranges;
  const int range = (int)(blockIdx.x - unit * ranges);
  pdl_launch_dependents();
  const Unit u = find_unit(p, unit, range == 0 && threadIdx.x == 0);
  if (u.count < 0) return;  // the whole cluster
  const int heads = min(p.group - u.part * kRows, kRows);
  const int head0 = u.h * p.group + u.part * kRows;
  const int begin = (int)((int64_t)u.count * range / ranges);
  const int end = (int)((int64_t)u.count * (range + 1) / ranges);

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
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          x[nt][i][e] = hd < heads ? to_f32(src[e]) : 0.f;
          big = fmaxf(big, fabsf(x[nt][i][e]));
        }
      }
    float down = 1.f;
    if constexpr (kPg == kF8) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, d));
      if (big > 16384.f && big < INFINITY) {
        const int ex = ilogbf(big) - 13;
        down = exp2f((float)-ex);
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

  uint4 kr[2][Tr::kKChunks];
  uint32_t vr[4][Tr::kVChunks][Tr::kVBytes / 4];
  constexpr int64_t kPageBytes = kBS * (int64_t)Tr::kRowBytes;
  const uint8_t* kbase = static_cast<const uint8_t*>(p.k_cache) + (int64_t)u.h * kPageBytes;
  const uint8_t* vbase = static_cast<const uint8_t*>(p.v_cache) + (int64_t)u.h * kPageBytes;
  const int64_t block_bytes = kPageBytes * p.num_kv_heads;
  const int koff = r * Tr::kRowBytes + c * 16;

  // keys of a page up to the token's position
  auto page_keys = [&](const Entry& e) {
    return e.phys < 0 ? 0 : min(kBS, u.pos - e.block * kBS + 1);
  };
  auto load_k = [&](const Entry& e) {
    const uint8_t* src = kbase + (int64_t)max(e.phys, 0) * block_bytes + koff;
    const bool on = e.phys >= 0;
#pragma unroll
    for (int i = 0; i < Tr::kKChunks; ++i) {
      kr[0][i] = kr[1][i] = make_uint4(0, 0, 0, 0);
      if (on) {
        kr[0][i] = __ldg(reinterpret_cast<const uint4*>(src + 64 * i));
        kr[1][i] = __ldg(reinterpret_cast<const uint4*>(src + 8 * Tr::kRowBytes + 64 * i));
      }
    }
  };
  // a row past the position holds nothing yet (its bits may be anything): 0
  auto load_v = [&](const Entry& e) {
    const uint8_t* src =
        vbase + (int64_t)max(e.phys, 0) * block_bytes + r * Tr::kVBytes;
    const int keys = page_keys(e);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int key = 2 * c + (j & 1) + 8 * (j >> 1);
#pragma unroll
      for (int i = 0; i < Tr::kVChunks; ++i) {
        const uint8_t* at = src + key * Tr::kRowBytes + i * 8 * Tr::kVBytes;
        if constexpr (Tr::kVBytes == 16) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (key < keys) v = __ldg(reinterpret_cast<const uint4*>(at));
          vr[j][i][0] = v.x; vr[j][i][1] = v.y; vr[j][i][2] = v.z; vr[j][i][3] = v.w;
        } else {
          uint2 v = make_uint2(0, 0);
          if (key < keys) v = __ldg(reinterpret_cast<const uint2*>(at));
          vr[j][i][0] = v.x; vr[j][i][1] = v.y;
        }
      }
    }
  };

  // the warp's entries, 32 at a time: begin + warp, + kWarps, ...
  const int mine = end - begin > warp ? (end - begin - warp + kWarps - 1) / kWarps : 0;
  Entry held{0, -1};
  auto entry = [&](int i) {  // the warp's entry i, in order
    if ((i & 31) == 0) {
      const int at = begin + warp + (i + lane) * kWarps;
      held = Entry{0, -1};
      if (i + lane < mine) held = list_entry(p, u, at);
    }
    // one lane asks a later page into L2: loads in flight beyond the registers
    if (kAhead > 0 && lane == ((i + kAhead) & 31) && lane >= kAhead && held.phys >= 0) {
      bulk_prefetch_l2(kbase + held.phys * block_bytes, (uint32_t)kPageBytes);
      bulk_prefetch_l2(vbase + held.phys * block_bytes, (uint32_t)kPageBytes);
    }
    return Entry{__shfl_sync(~0u, held.block, i & 31), __shfl_sync(~0u, held.phys, i & 31)};
  };
  Entry cur{0, -1};
  if (mine > 0) {
    cur = entry(0);
    load_k(cur);
    load_v(cur);
  }
  for (int i = 0; i < mine; ++i) {
    const int keys = page_keys(cur);
    // S^T = K Q^T: keys r and r + 8, heads 2c and 2c + 1
    float s[kNT][4];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
    for (int ch = 0; ch < Tr::kKChunks; ++ch) {
      const uint32_t w0[4] = {kr[0][ch].x, kr[0][ch].y, kr[0][ch].z, kr[0][ch].w};
      const uint32_t w1[4] = {kr[1][ch].x, kr[1][ch].y, kr[1][ch].z, kr[1][ch].w};
      if constexpr (kPg == kF8) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a[4];
          e4m3x4_to_f16x2x2(w0[w], a[0], a[2]);
          e4m3x4_to_f16x2x2(w1[w], a[1], a[3]);
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
            mma16816<false>(s[nt], a, qw[nt][ch][2 * w], qw[nt][ch][2 * w + 1]);
        }
      } else {
#pragma unroll
        for (int w = 0; w < 4; w += 2) {
          const uint32_t a[4] = {w0[w], w1[w], w0[w + 1], w1[w + 1]};
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
            mma16816<kBF>(s[nt], a, qw[nt][ch][w], qw[nt][ch][w + 1]);
        }
      }
    }
    Entry next{0, -1};
    if (i + 1 < mine) {
      next = entry(i + 1);
      load_k(next);
    }
    // softmax over the page
    uint32_t pb[kNT][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[nt][j] = r + 8 * (j >> 1) < keys ? s[nt][j] * score_scale : -INFINITY;
      float mx[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mx[j] = fmaxf(s[nt][j], s[nt][j + 2]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) mx[j] = fmaxf(mx[j], __shfl_xor_sync(~0u, mx[j], d));
        mx[j] = fmaxf(mx[j], m[nt][j]);
      }
      if (__any_sync(~0u, mx[0] > m[nt][0] || mx[1] > m[nt][1])) {
        float al[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          al[j] = mx[j] == -INFINITY ? 1.f : exp2f(m[nt][j] - mx[j]);
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
      const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
      const float m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
      const float p0 = exp2f(s[nt][0] - m0), p1 = exp2f(s[nt][1] - m1);
      const float p2 = exp2f(s[nt][2] - m0), p3 = exp2f(s[nt][3] - m1);
      l[nt][0] += p0 + p2;
      l[nt][1] += p1 + p3;
      // keys as rows -> heads as rows: the second product's operand
      pb[nt][0] = transpose8x8(pack2<kBF>(p0, p1));
      pb[nt][1] = transpose8x8(pack2<kBF>(p2, p3));
    }
    // O^T += V^T P^T: channels as rows
#pragma unroll
    for (int ch = 0; ch < Tr::kVChunks; ++ch)
#pragma unroll
      for (int w = 0; w < Tr::kVBytes / 4; ++w) {
        const uint32_t a0 = vr[0][ch][w], a1 = vr[1][ch][w];
        const uint32_t a2 = vr[2][ch][w], a3 = vr[3][ch][w];
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
              mma16816<false>(acc[nt][(ch * (Tr::kVBytes / 4) + w) * 2 + k], a, pb[nt][0],
                              pb[nt][1]);
          }
        } else {
          const uint32_t a[4] = {__byte_perm(a0, a1, 0x5410), __byte_perm(a0, a1, 0x7632),
                                 __byte_perm(a2, a3, 0x5410), __byte_perm(a2, a3, 0x7632)};
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
            mma16816<kBF>(acc[nt][ch * (Tr::kVBytes / 4) + w], a, pb[nt][0], pb[nt][1]);
        }
      }
    if (i + 1 < mine) load_v(next);
    cur = next;
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
  // the CTA's result into the place of warp 0's (each thread reads and writes
  // its own elements), then the cluster's from all of its CTAs
  for (int i = threadIdx.x; i < heads * kD; i += kThreads) {
    const int hd = i / kD, d = i - hd * kD;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][hd]);
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      a += (s_m[w][hd] == -INFINITY ? 0.f : exp2f(s_m[w][hd] - mx)) * s_acc[w][hd][d];
    s_acc[0][hd][d] = a;
  }
  __shared__ float s_ml[kRows][2];
  if (threadIdx.x < heads) {
    const int hd = threadIdx.x;
    float mx = -INFINITY, ls = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][hd]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      ls += (s_m[w][hd] == -INFINITY ? 0.f : exp2f(s_m[w][hd] - mx)) * s_l[w][hd];
    s_ml[hd][0] = mx;
    s_ml[hd][1] = ls;
  }
  cg::cluster_group cl = cg::this_cluster();
  if (p.cluster > 1) cl.sync(); else __syncthreads();
  const int rank = p.cluster > 1 ? (int)cl.block_rank() : 0;
  for (int i = rank * kThreads + threadIdx.x; i < heads * kD; i += p.cluster * kThreads) {
    const int hd = i / kD, d = i - hd * kD;
    float mx = s_ml[hd][0], ls = s_ml[hd][1], a = s_acc[0][hd][d];
    if (p.cluster > 1) {
      mx = -INFINITY;
      for (int c2 = 0; c2 < p.cluster; ++c2)
        mx = fmaxf(mx, *cl.map_shared_rank(&s_ml[hd][0], c2));
      ls = a = 0.f;
      for (int c2 = 0; c2 < p.cluster; ++c2) {
        const float ms = *cl.map_shared_rank(&s_ml[hd][0], c2);
        const float f = ms == -INFINITY ? 0.f : exp2f(ms - mx);
        ls += f * *cl.map_shared_rank(&s_ml[hd][1], c2);
        a += f * *cl.map_shared_rank(&s_acc[0][hd][d], c2);
      }
    }
    if (p.splits == 1) {
      static_cast<TQ*>(p.out)[(u.t * p.num_q_heads + head0 + hd) * kD + d] =
          from_f32<TQ>(ls == 0.f ? 0.f : a / ls * p.v_scale);
    } else {
      const int64_t row = (unit * p.splits + range / p.cluster) * p.head_rows + hd;
      p.part[row * kD + d] = a;
      if (d == 0) {
        p.part_ml[2 * row] = mx;
        p.part_ml[2 * row + 1] = ls;
      }
    }
  }
  if (p.cluster > 1) cl.sync();  // the others may still read this CTA's memory
}

// Join a unit's splits in order: one warp per (unit, query head).
template <typename TQ, int kD>
__global__ void __launch_bounds__(kThreads) selected_join_kernel(const SelParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t units = p.s.num_tokens * p.num_kv_heads * p.head_parts;
  const int64_t unit = item / p.head_rows;
  const int hd = (int)(item - unit * p.head_rows);
  if (unit >= units) return;
  const Unit u = find_unit(p, unit, false);
  pdl_wait();  // the splits' results
  if (u.count < 0 || hd >= min(p.group - u.part * p.head_rows, p.head_rows)) return;
  const int64_t row0 = unit * p.splits * p.head_rows + hd;
  float mx = -INFINITY;
  for (int s = 0; s < p.splits; ++s)
    mx = fmaxf(mx, p.part_ml[2 * (row0 + (int64_t)s * p.head_rows)]);
  float a[kD / 32] = {}, ls = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const int64_t row = row0 + (int64_t)s * p.head_rows;
    const float ms = p.part_ml[2 * row];
    const float f = ms == -INFINITY ? 0.f : exp2f(ms - mx);
    ls += f * p.part_ml[2 * row + 1];
#pragma unroll
    for (int k = 0; k < kD / 32; ++k) a[k] += f * p.part[row * kD + lane + 32 * k];
  }
  TQ* out = static_cast<TQ*>(p.out) +
            (u.t * p.num_q_heads + u.h * p.group + u.part * p.head_rows + hd) * kD;
#pragma unroll
  for (int k = 0; k < kD / 32; ++k)
    out[lane + 32 * k] = from_f32<TQ>(ls == 0.f ? 0.f : a[k] / ls * p.v_scale);
}

cudaError_t launched() {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename TQ, typename TP>
cudaError_t launch_generic(SelParams& p, int head_dim, cudaStream_t stream) {
  p.head_parts = 1;
  const int64_t grid = p.s.num_tokens * p.num_q_heads;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  if (head_dim == 128)
    selected_generic_kernel<TQ, TP, 128><<<(unsigned)grid, kThreads, 0, stream>>>(p);
  else
    selected_generic_kernel<TQ, TP, 64><<<(unsigned)grid, kThreads, 0, stream>>>(p);
  return launched();
}

template <typename TQ, int kPg, int kD>
cudaError_t launch_mma_d(const SelParams& p, int64_t units, cudaStream_t stream) {
  const int64_t grid = units * p.cluster * p.splits;
  const int64_t join = (units * p.head_rows + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffll || join > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)p.cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
  cudaError_t e = p.head_rows == 8
                      ? cudaLaunchKernelEx(&cfg, selected_kernel<TQ, kPg, kD, 1>, p)
                      : cudaLaunchKernelEx(&cfg, selected_kernel<TQ, kPg, kD, 2>, p);
  if (e != cudaSuccess) return e;
  count_launch();
  if (p.splits == 1) return cudaSuccess;
  cfg.gridDim = dim3((unsigned)join);
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, selected_join_kernel<TQ, kD>, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename TQ, int kPg>
cudaError_t launch_mma(const SelParams& p, int head_dim, int64_t units,
                       cudaStream_t stream) {
  return head_dim == 128 ? launch_mma_d<TQ, kPg, 128>(p, units, stream)
                         : launch_mma_d<TQ, kPg, 64>(p, units, stream);
}

}  // namespace

SelectedPlan make_selected_plan(int64_t num_tokens, int num_q_heads, int num_kv_heads,
                                int head_dim, int max_selected, int num_sms) {
  SelectedPlan pl{};
  const int group = num_q_heads / num_kv_heads;
  pl.head_rows = group <= 8 ? 8 : 16;
  pl.head_parts = (group + pl.head_rows - 1) / pl.head_rows;
  pl.units = num_tokens * num_kv_heads * pl.head_parts;
  // Ranges per list: until the grid is kSelWaves CTAs per SM, of two pages per
  // warp at least.  Up to 8 (a portable cluster) are joined through the
  // cluster's shared memory; beyond that, clusters through the workspace.
  const int64_t want = (int64_t)kSelWaves * num_sms;
  const int64_t most = std::max(1, max_selected / (2 * kWarps));
  int64_t ranges = pl.units > 0 ? (want + pl.units - 1) / pl.units : 1;
  ranges = std::max<int64_t>(1, std::min(ranges, most));
  pl.cluster = 1;
  while (pl.cluster < 8 && pl.cluster < ranges) pl.cluster *= 2;
  if (pl.cluster > most) pl.cluster /= 2;
  pl.splits = ranges > 8 ? (int)((ranges + 7) / 8) : 1;
  pl.bytes = pl.splits == 1 ? 0
                            : pl.units * pl.splits * pl.head_rows * (head_dim + 2) *
                                  (int64_t)sizeof(float);
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
  p.head_parts = plan.head_parts;
  p.head_rows = plan.head_rows;
  p.cluster = plan.cluster;
  p.splits = plan.splits;
  p.selected = a.selected;
  p.num_selected = a.num_selected;
  p.max_selected = a.max_selected;
  p.scale = a.scale;
  const bool scaled = a.cache_dtype == PA_FP8_E4M3 || a.cache_dtype == PA_NVFP4;
  p.k_scale = scaled ? a.k_scale : 1.0f;
  p.v_scale = scaled ? a.v_scale : 1.0f;
  p.out = a.out;
  p.part = static_cast<float*>(a.workspace);
  p.part_ml =
      p.part + plan.units * plan.splits * plan.head_rows * (int64_t)a.head_dim;
  const bool bf = a.q_dtype == PA_BF16;
  switch (a.cache_dtype) {
    case PA_F32: return launch_generic<float, F32Page>(p, a.head_dim, stream);
    case PA_F16: return launch_mma<__half, kH16>(p, a.head_dim, plan.units, stream);
    case PA_BF16:
      return launch_mma<__nv_bfloat16, kB16>(p, a.head_dim, plan.units, stream);
    case PA_FP8_E4M3:
      return bf ? launch_mma<__nv_bfloat16, kF8>(p, a.head_dim, plan.units, stream)
                : launch_mma<__half, kF8>(p, a.head_dim, plan.units, stream);
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
