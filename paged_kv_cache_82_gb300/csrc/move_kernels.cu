// move_kernels.cu -- blocks copied and tokens moved in the caches of all layers at
// once (pa_copy_blocks_layers, pa_move_tokens).
//
// Both only move bytes, 2 x what they copy, and are bound by HBM; what they add to
// the single layer's pa_copy_blocks is one launch instead of one per layer, and a
// count that the host need not know.
#include "pa_beam.h"
#include "pa_common.cuh"

namespace pa {
namespace {

// ---- blocks --------------------------------------------------------------------
// A CTA copies pieces of up to 32 KB, eight 16-byte loads of each thread in flight: 24
// blocks x 32 layers of bf16 16.9 us, 500 x 80 of E4M3 395 us = 6.6 TB/s (98 % of a plain
// copy's rate; with four loads and eight CTAs per SM 16.8 and 420).  Smaller blocks have
// fewer threads, not fewer loads of each: 200 blocks x 32 layers of INT4, 8 heads of 64,
// 18.8 us (floor 17.3; with a thread to a load 40.7, to four 21.1); of 8 heads of 64 E4M3
// channels 32.4 (30.8; 48.6, 33.6).
constexpr int kCopyLoads = 8;
constexpr int kMaxCopyThreads = 256;  // fewer where a block is smaller than 32 KB
constexpr int kCopyCtasPerSm = 64;    // CTAs of a grid: more than are resident, for a short
                                      // last wave

struct CopyK {
  char* k;
  char* v;
  int64_t k_layer, v_layer;  // bytes
  int64_t num_blocks;
  int64_t block_vecs;  // 16-byte vectors of a block of one layer's K (or V)
  int pieces;          // of a block
  int num_layers;
  const int64_t* mapping;
  int64_t max_pairs;
  const int32_t* num_pairs;  // null: max_pairs
  unsigned* err;
};

__global__ void __launch_bounds__(kMaxCopyThreads) copy_layers_kernel(CopyK p) {
  const int threads = blockDim.x;
  int64_t pairs = p.max_pairs;
  if (p.num_pairs) {
    pairs = *p.num_pairs;
    if (pairs < 0 || pairs > p.max_pairs) {
      if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(p.err, PA_DEV_ERR_METADATA);
      pairs = pairs < 0 ? 0 : p.max_pairs;
    }
  }
  const int per_pair = p.num_layers * 2 * p.pieces;
  const int64_t items = pairs * per_pair;
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const int64_t pair = i / per_pair;
    int rest = (int)(i - pair * per_pair);
    const int piece = rest % p.pieces;
    rest /= p.pieces;
    const bool is_v = rest & 1;
    const int layer = rest >> 1;
    const int64_t src = __ldg(p.mapping + 2 * pair), dst = __ldg(p.mapping + 2 * pair + 1);
    if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_blocks) {
      if (threadIdx.x == 0) flag_error(p.err, PA_DEV_ERR_BLOCK_ID);
      continue;
    }
    uint4* base = reinterpret_cast<uint4*>(is_v ? p.v + layer * p.v_layer
                                                : p.k + layer * p.k_layer);
    const uint4* from = base + src * p.block_vecs;
    uint4* to = base + dst * p.block_vecs;
    const int64_t first = (int64_t)piece * (threads * kCopyLoads) + threadIdx.x;
    uint4 x[kCopyLoads];
#pragma unroll
    for (int j = 0; j < kCopyLoads; ++j)
      if (first + j * threads < p.block_vecs) x[j] = __ldcs(from + first + j * threads);
#pragma unroll
    for (int j = 0; j < kCopyLoads; ++j)
      if (first + j * threads < p.block_vecs) to[first + j * threads] = x[j];
  }
}

// ---- tokens --------------------------------------------------------------------
// A row's moves may overwrite what earlier ones of the row have read, so they are
// done in order.  Each channel of each head of each layer has an order of its own: a
// warp takes slices of heads' channels through all moves of a row, and no warp waits
// for another: 8 prompts cut from 4K-8K to half, 16 layers of bf16, 488 us = 6.4 TB/s
// (94 % of a plain copy's rate).  Reading ahead is always right (no destination is a later
// source), so a warp keeps kStages steps of loads in flight, through shared memory, and
// writes a step once it and those before it have landed.
constexpr int kMoveWarps = 4;
constexpr int kStages = 8;
constexpr int kStageLoads = 4;    // 16-byte loads of a lane in one step, at most
constexpr int kMoveCtasPerSm = 3;  // by shared memory
constexpr int kAhead = 4;          // steps whose slots are looked up ahead
constexpr int kScaleLoads = 8;

struct MoveK {
  char* k;
  char* v;
  int64_t k_layer, v_layer;  // bytes
  int64_t num_slots;
  int heads, num_layers, num_rows;
  int64_t page_bytes;
  int row_bytes;    // of a token's channels (codes) in a page
  int scale_bytes;  // of a token's scales behind them (4-bit pages), 0: none
  int per_warp;     // slices that a warp takes, one after another
  int row_warps;    // warps of a row
  const int64_t* src;
  const int64_t* dst;
  const int32_t* num_moves;
  int64_t max_moves;
  unsigned* err;
};

// A place in a layer's cache in units of 32 bytes, which every token's channels (codes)
// start on; kNowhere: no move.
constexpr uint32_t kNowhere = 0xffffffffu;
static_assert(PA_PAGE_BYTES(PA_INT4, 64) % 32 == 0 && PA_PAGE_BYTES(PA_NVFP4, 64) % 32 == 0,
              "pages start on 32 bytes");

template <int kTokens>
struct MoveRing {  // a warp's steps in flight
  uint4 data[kStages][kStageLoads][32];
  uint32_t dst[kStages][kTokens < 32 ? 32 : kTokens];  // each token's place
};

// The slices [u, u_end) of a row's heads (a layer's K, then its V, head by head), of
// 2^kLg lanes each.  Few warps share an SM where there are few heads, so that a step's
// instructions count: places are 32-bit, and the loops' bounds known.
template <int kLg>
__device__ __forceinline__ void move_slices(const MoveK& p, char* shared, int u, int u_end,
                                            const int64_t* src, const int64_t* dst, int n,
                                            bool reports) {
  constexpr int kPer = 32 >> kLg;               // tokens of one load
  constexpr int kTokens = kPer * kStageLoads;   // of one step
  constexpr int kMine = (kTokens + 31) / 32;    // looked up by a lane
  auto& ring = *reinterpret_cast<MoveRing<kTokens>*>(shared);
  const int lane = threadIdx.x & 31, token = lane >> kLg;
  const int column = (lane & ((1 << kLg) - 1)) * 16;
  const int slices = p.row_bytes >> (kLg + 4);
  const uint32_t block = (uint32_t)(p.heads * p.page_bytes / 32);
  const uint32_t line = (uint32_t)(p.row_bytes / 32);
  // The slots of the next kAhead steps, in registers: step i's at i % kAhead, loaded when
  // step i - kAhead has used them.
  int64_t from[kAhead][kMine], to[kAhead][kMine];
  int listed = 0;        // first move of the next step to look up
  int j = 0;             // and of the next step to issue
  char* base = nullptr;  // of that step's slice; this lane's column of it
  auto base_of = [&](int unit) {
    const int slice = unit % slices, rest = unit / slices, head = rest % p.heads;
    const int layer = rest / p.heads;
    return (layer & 1 ? p.v + (layer >> 1) * p.v_layer : p.k + (layer >> 1) * p.k_layer) +
           head * p.page_bytes + slice * (16 << kLg) + column;
  };
  auto look_up = [&](int64_t (&a)[kMine], int64_t (&b)[kMine]) {
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const int i = m * 32 + lane;
      const bool on = i < kTokens && listed + i < n;
      a[m] = on ? __ldg(src + listed + i) : -1;
      b[m] = on ? __ldg(dst + listed + i) : -1;
    }
    listed += kTokens;
    if (listed >= n) listed = 0;  // (the same list for the next slice)
  };
  auto place = [&](int64_t slot) {
    return (uint32_t)(slot / kBS) * block + (uint32_t)(slot % kBS) * line;
  };
  auto issue = [&](int stage, int64_t (&sf)[kMine], int64_t (&st)[kMine]) {
    if (u < u_end) {
      uint32_t a[kMine];
#pragma unroll
      for (int m = 0; m < kMine; ++m) {
        const bool in = sf[m] < p.num_slots && st[m] < p.num_slots;
        if (!in && reports) flag_error(p.err, PA_DEV_ERR_SLOT);
        const bool moves = in && sf[m] >= 0 && st[m] >= 0 && sf[m] != st[m];
        a[m] = moves ? place(sf[m]) : kNowhere;
        ring.dst[stage][m * 32 + lane] = moves ? place(st[m]) : kNowhere;
      }
      look_up(sf, st);
#pragma unroll
      for (int e = 0; e < kStageLoads; ++e) {
        const uint32_t at = __shfl_sync(~0u, a[e * kPer / 32], (e * kPer & 31) + token);
        if (at != kNowhere)
          copy_async16(smem_u32(&ring.data[stage][e][lane]), base + (uint64_t)at * 32);
      }
      j += kTokens;
      if (j >= n) {
        j = 0;
        if (++u < u_end) base = base_of(u);
      }
    }
    async_commit();
  };
  const int64_t total = (int64_t)(u_end - u) * ((n + kTokens - 1) / kTokens);
  base = base_of(u);
  char* done_base = base;  // the same for the step to be written
  int done_u = u, done_j = 0;
#pragma unroll
  for (int i = 0; i < kAhead; ++i) look_up(from[i], to[i]);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i, from[i % kAhead], to[i % kAhead]);
#pragma unroll 1
  for (int64_t done = 0; done < total; done += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int stage = (int)((done + k) % kStages);
      issue((stage + kStages - 1) % kStages, from[(k + kStages - 1) % kAhead],
            to[(k + kStages - 1) % kAhead]);
      async_wait<kStages - 1>();
      __syncwarp();  // the step has landed, for every lane
      if (done + k < total) {
#pragma unroll
        for (int e = 0; e < kStageLoads; ++e) {
          const uint32_t at = ring.dst[stage][e * kPer + token];
          if (at != kNowhere)
            *reinterpret_cast<uint4*>(done_base + (uint64_t)at * 32) = ring.data[stage][e][lane];
        }
        done_j += kTokens;
        if (done_j >= n) {
          done_j = 0;
          if (++done_u < u_end) done_base = base_of(done_u);
        }
      }
      __syncwarp();  // its places are free
    }
  }
}

// The scales of one head of 4-bit pages: 4 or 8 bytes of a token, a lane to a token.
template <typename Vec>
__device__ __forceinline__ void move_scales(const MoveK& p, char* base, int head,
                                            const int64_t* src, const int64_t* dst, int n) {
  const int lane = threadIdx.x & 31;
  auto place = [&](int64_t slot) {
    return reinterpret_cast<Vec*>(base + ((slot / kBS) * p.heads + head) * p.page_bytes +
                                  kBS * p.row_bytes) + slot % kBS;
  };
  for (int j0 = 0; j0 < n; j0 += 32 * kScaleLoads) {
    int64_t from[kScaleLoads], to[kScaleLoads];
    Vec x[kScaleLoads];
#pragma unroll
    for (int e = 0; e < kScaleLoads; ++e) {
      const int j = j0 + e * 32 + lane;
      from[e] = j < n ? __ldg(src + j) : -1;
      to[e] = j < n ? __ldg(dst + j) : -1;
    }
#pragma unroll
    for (int e = 0; e < kScaleLoads; ++e) {
      if (from[e] < 0 || from[e] >= p.num_slots || to[e] >= p.num_slots) to[e] = -1;
      if (to[e] >= 0) x[e] = __ldcg(place(from[e]));
    }
    __syncwarp();  // all of the step is read
#pragma unroll
    for (int e = 0; e < kScaleLoads; ++e)
      if (to[e] >= 0) *place(to[e]) = x[e];
    __syncwarp();
  }
}

template <int kLg>
__global__ void __launch_bounds__(32 * kMoveWarps, kMoveCtasPerSm)
    move_tokens_kernel(MoveK p) {
  extern __shared__ __align__(16) char shared[];
  const int warp = threadIdx.x >> 5;
  const int64_t w = (int64_t)blockIdx.x * kMoveWarps + warp;
  const int64_t row = w / p.row_warps;
  if (row >= p.num_rows) return;
  const int part = (int)(w - row * p.row_warps);
  const int n = __ldg(p.num_moves + row);
  if (n < 0 || n > p.max_moves) {
    if (part == 0 && (threadIdx.x & 31) == 0) flag_error(p.err, PA_DEV_ERR_METADATA);
    return;
  }
  if (n == 0) return;
  const int64_t* src = p.src + row * p.max_moves;
  const int64_t* dst = p.dst + row * p.max_moves;
  const int heads = p.num_layers * 2 * p.heads;
  const int data = heads * (p.row_bytes >> (kLg + 4));
  const int first = part * p.per_warp, end = first + p.per_warp;
  if (first < data)
    move_slices<kLg>(p, shared + warp * sizeof(MoveRing<kStageLoads * (32 >> kLg)>), first,
                     min(end, data), src, dst, n, part == 0);
  if (p.scale_bytes)
    for (int u = max(first, data); u < min(end, data + heads); ++u) {
      const int head = (u - data) % p.heads, layer = (u - data) / p.heads;
      char* base = layer & 1 ? p.v + (layer >> 1) * p.v_layer : p.k + (layer >> 1) * p.k_layer;
      if (p.scale_bytes == 4)
        move_scales<uint32_t>(p, base, head, src, dst, n);
      else
        move_scales<uint2>(p, base, head, src, dst, n);
    }
}

template <int kLg>
cudaError_t launch_moves(const MoveK& p, unsigned ctas, cudaStream_t stream) {
  constexpr size_t kSmem = kMoveWarps * sizeof(MoveRing<kStageLoads * (32 >> kLg)>);
  static_assert(kMoveCtasPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
  cudaError_t e = cudaFuncSetAttribute(move_tokens_kernel<kLg>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  move_tokens_kernel<kLg><<<ctas, 32 * kMoveWarps, kSmem, stream>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

cudaError_t launch_copy_blocks_layers(const LayerCaches& c, int64_t block_bytes,
                                      const int64_t* block_mapping, int64_t max_pairs,
                                      const int32_t* num_pairs, int num_sms, unsigned* err,
                                      cudaStream_t stream) {
  CopyK p{};
  p.k = static_cast<char*>(c.k);
  p.v = static_cast<char*>(c.v);
  p.k_layer = c.k_layer_bytes;
  p.v_layer = c.v_layer_bytes;
  p.num_blocks = c.num_blocks;
  p.block_vecs = block_bytes / 16;
  const int64_t warps = (p.block_vecs + 32 * kCopyLoads - 1) / (32 * kCopyLoads);
  const int threads = warps * 32 < kMaxCopyThreads ? (int)warps * 32 : kMaxCopyThreads;
  p.pieces = (int)((p.block_vecs + threads * kCopyLoads - 1) / (threads * kCopyLoads));
  p.num_layers = c.num_layers;
  p.mapping = block_mapping;
  p.max_pairs = max_pairs;
  p.num_pairs = num_pairs;
  p.err = err;
  const int64_t items = max_pairs * c.num_layers * 2 * p.pieces;
  const int64_t most = (int64_t)num_sms * kCopyCtasPerSm;
  copy_layers_kernel<<<(unsigned)(items < most ? items : most), threads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t launch_move_tokens(const LayerCaches& c, const int64_t* src_slots,
                               const int64_t* dst_slots, const int32_t* num_moves,
                               int num_rows, int64_t max_moves, int num_sms, unsigned* err,
                               cudaStream_t stream) {
  MoveK p{};
  p.k = static_cast<char*>(c.k);
  p.v = static_cast<char*>(c.v);
  p.k_layer = c.k_layer_bytes;
  p.v_layer = c.v_layer_bytes;
  p.num_slots = c.num_blocks * kBS;
  p.heads = c.num_kv_heads;
  p.num_layers = c.num_layers;
  p.num_rows = num_rows;
  const int D = c.head_dim;
  p.row_bytes = c.dtype == PA_F32           ? 4 * D
                : c.dtype == PA_FP8_E4M3    ? D
                : is_4bit(c.dtype)          ? D / 2
                                            : 2 * D;
  p.scale_bytes = c.dtype == PA_INT4 ? 4 : c.dtype == PA_NVFP4 ? D / 16 : 0;
  p.page_bytes = (int64_t)kBS * (p.row_bytes + p.scale_bytes);
  p.src = src_slots;
  p.dst = dst_slots;
  p.num_moves = num_moves;
  p.max_moves = max_moves;
  p.err = err;
  // A slice is a head's whole token; half of it and so on, down to 128 bytes (DRAM reads
  // lines of that length: with 64 the moves of 8 prompts of 4K-8K in 16 layers took 787 us,
  // with 128 488, with 256 534), while there are fewer than four slices to a resident warp;
  // and down to a sector while there are fewer than one (a prompt of 32K, 8 heads of 64 E4M3
  // channels in 32 layers: 157 -> 124 us).  A warp takes several slices of a row, one
  // after another, where there are more than four waves of warps for, two if lists are
  // short: its first loads wait once, not once per slice (64 lists of 6 tokens in 32
  // layers: one wave 27.5 us, two 21.4, four 22.3).
  const int64_t resident = (int64_t)num_sms * kMoveCtasPerSm * kMoveWarps;
  const int64_t heads = (int64_t)c.num_layers * 2 * c.num_kv_heads;
  int lg = 0;
  while ((16 << lg) < p.row_bytes) ++lg;
  auto slices = [&]() { return num_rows * heads * (p.row_bytes >> (lg + 4)); };
  while (lg > 3 && slices() < 4 * resident) --lg;
  while (lg > 1 && slices() < resident) --lg;
  const int64_t units = heads * ((p.row_bytes >> (lg + 4)) + (p.scale_bytes ? 1 : 0));
  const int64_t waves = max_moves <= 64 ? 2 : 4;
  int64_t per_warp = (num_rows * units + waves * resident - 1) / (waves * resident);
  if (per_warp > 32) per_warp = 32;
  if (per_warp > units) per_warp = units;
  p.per_warp = (int)per_warp;
  p.row_warps = (int)((units + per_warp - 1) / per_warp);
  const int64_t ctas = ((int64_t)num_rows * p.row_warps + kMoveWarps - 1) / kMoveWarps;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  switch (lg) {
    case 1: return launch_moves<1>(p, (unsigned)ctas, stream);
    case 2: return launch_moves<2>(p, (unsigned)ctas, stream);
    case 3: return launch_moves<3>(p, (unsigned)ctas, stream);
    case 4: return launch_moves<4>(p, (unsigned)ctas, stream);
    default: return launch_moves<5>(p, (unsigned)ctas, stream);
  }
}

}  // namespace pa
