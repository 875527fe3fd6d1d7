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

constexpr int kThreads = 256;

// ---- blocks --------------------------------------------------------------------
// A CTA copies pieces of kPiece bytes: a quarter of it in flight per 16-byte load of
// its threads.
constexpr int kCopyLoads = 4;
constexpr int kPieceVecs = kThreads * kCopyLoads;

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

__global__ void __launch_bounds__(kThreads) copy_layers_kernel(CopyK p) {
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
    const int64_t first = (int64_t)piece * kPieceVecs + threadIdx.x;
    uint4 x[kCopyLoads];
#pragma unroll
    for (int j = 0; j < kCopyLoads; ++j)
      if (first + j * kThreads < p.block_vecs) x[j] = __ldcs(from + first + j * kThreads);
#pragma unroll
    for (int j = 0; j < kCopyLoads; ++j)
      if (first + j * kThreads < p.block_vecs) to[first + j * kThreads] = x[j];
  }
}

// ---- tokens --------------------------------------------------------------------
// A row's moves may overwrite what earlier ones of the row have read, so they are
// done in order.  Each channel of each head of each layer has an order of its own: a
// warp takes a slice of one head's channels through all moves of a row, a step of
// many tokens at a time, all of a step read before any of it is written.  No warp
// waits for another.
constexpr int kMoveLoads = 8;  // of a lane in one step
constexpr int kMoveWarps = kThreads / 32;

struct MoveK {
  char* k;
  char* v;
  int64_t k_layer, v_layer;  // bytes
  int64_t num_slots;
  int heads, num_layers, num_rows;
  int64_t page_bytes;
  int row_bytes;    // of a token's channels (codes) in a page
  int scale_bytes;  // of a token's scales behind them (4-bit pages), 0: none
  int lanes_log2;   // lanes of a slice: 16 bytes each
  int slices;       // slices of a token, the scales' included
  const int64_t* src;
  const int64_t* dst;
  const int32_t* num_moves;
  int64_t max_moves;
  unsigned* err;
};

// One slice through the moves of a row: 2^lg lanes of a Vec to a token.
template <typename Vec>
__device__ __forceinline__ void move_slice(const MoveK& p, char* base, int head,
                                           int64_t offset, int token_bytes, int lg,
                                           const int64_t* src, const int64_t* dst, int n,
                                           bool reports) {
  const int lane = threadIdx.x & 31;
  const int per = 32 >> lg;  // tokens of one load
  const int64_t mine = offset + (int64_t)(lane & ((1 << lg) - 1)) * sizeof(Vec);
  auto place = [&](int64_t slot) {
    return base + ((slot / kBS) * p.heads + head) * p.page_bytes +
           (slot % kBS) * token_bytes + mine;
  };
  for (int j0 = lane >> lg; j0 - (lane >> lg) < n; j0 += per * kMoveLoads) {
    int64_t from[kMoveLoads], to[kMoveLoads];
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e) {
      const int j = j0 + e * per;
      from[e] = j < n ? __ldg(src + j) : -1;
      to[e] = j < n ? __ldg(dst + j) : -1;
    }
    Vec x[kMoveLoads];
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e) {
      if (from[e] >= p.num_slots || to[e] >= p.num_slots) {
        if (reports) flag_error(p.err, PA_DEV_ERR_SLOT);
        from[e] = -1;
      }
      if (from[e] < 0 || from[e] == to[e]) to[e] = -1;
      if (to[e] >= 0) x[e] = __ldcg(reinterpret_cast<const Vec*>(place(from[e])));
    }
    __syncwarp();  // all of the step is read
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e)
      if (to[e] >= 0) *reinterpret_cast<Vec*>(place(to[e])) = x[e];
    __syncwarp();
  }
}

__global__ void __launch_bounds__(kThreads) move_tokens_kernel(MoveK p) {
  int64_t u = (int64_t)blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
  const int per_row = p.num_layers * 2 * p.heads * p.slices;
  const int64_t row = u / per_row;
  if (row >= p.num_rows) return;
  int rest = (int)(u - row * per_row);
  int n = __ldg(p.num_moves + row);
  const bool reports = rest == 0;
  if (n < 0 || n > p.max_moves) {
    if (reports && (threadIdx.x & 31) == 0) flag_error(p.err, PA_DEV_ERR_METADATA);
    return;
  }
  const int slice = rest % p.slices;
  rest /= p.slices;
  const int head = rest % p.heads;
  rest /= p.heads;
  const int layer = rest >> 1;
  char* base = rest & 1 ? p.v + layer * p.v_layer : p.k + layer * p.k_layer;
  const int64_t* src = p.src + row * p.max_moves;
  const int64_t* dst = p.dst + row * p.max_moves;
  const int slice_bytes = 16 << p.lanes_log2;
  const int data = p.row_bytes / slice_bytes;
  if (slice < data)
    move_slice<uint4>(p, base, head, (int64_t)slice * slice_bytes, p.row_bytes, p.lanes_log2,
                      src, dst, n, reports);
  else if (p.scale_bytes == 4)
    move_slice<uint32_t>(p, base, head, (int64_t)kBS * p.row_bytes, 4, 0, src, dst, n, false);
  else
    move_slice<uint2>(p, base, head, (int64_t)kBS * p.row_bytes, 8, 0, src, dst, n, false);
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
  p.pieces = (int)((p.block_vecs + kPieceVecs - 1) / kPieceVecs);
  p.num_layers = c.num_layers;
  p.mapping = block_mapping;
  p.max_pairs = max_pairs;
  p.num_pairs = num_pairs;
  p.err = err;
  // as many CTAs as stay resident (8 to an SM), fewer where there is less to do
  const int64_t items = max_pairs * c.num_layers * 2 * p.pieces;
  const int64_t most = (int64_t)num_sms * 8;
  copy_layers_kernel<<<(unsigned)(items < most ? items : most), kThreads, 0, stream>>>(p);
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
  // a warp to a head's whole token, in slices of 32 bytes (a sector) at least where
  // that leaves the SMs short of warps
  const int64_t heads = (int64_t)num_rows * c.num_layers * 2 * c.num_kv_heads;
  int lg = 0;
  while ((16 << lg) < p.row_bytes) ++lg;
  while (lg > 1 && heads * (p.row_bytes >> (lg + 4)) < (int64_t)num_sms * 16) --lg;
  p.lanes_log2 = lg;
  p.slices = (p.row_bytes >> (lg + 4)) + (p.scale_bytes ? 1 : 0);
  const int64_t ctas = (heads * p.slices + kMoveWarps - 1) / kMoveWarps;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  move_tokens_kernel<<<(unsigned)ctas, kThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace pa
