// fork_kernels.cu -- block tables, reference counts and the stack of free ids
// when rows take over other rows' blocks (pa_fork_blocks) or drop tokens
// (pa_compact_blocks).
//
// References.  extra_refs[b] counts a block's holders beyond the first; a count
// that falls below 0 frees the block.  All changes are integer additions, so
// their order does not matter:
//   fork:    an old row s that u new rows take over changes the count of each of
//            its blocks by u - 1 (nothing to do for u = 1);
//   compact: each entry dropped or replaced by a fresh block changes it by -1.
//
// Order.  Freed blocks go onto the stack in the order of the first released entry
// (row, column) that names them.  Which that is does not depend on timing: every
// released entry of a block whose count fell below 0 proposes INT_MIN + its place
// to the count itself by atomicMin; the lowest wins, and afterwards owns the push.
//
// A few MB at most are read (tables, counts), in four dependent passes over the
// released entries: latency bounds it, so the passes run in one cluster of CTAs
// with cluster barriers between them (a grid's barrier or a launch costs several
// of those), and a wide second kernel writes the tables and lists.
#include <cooperative_groups.h>
#include <limits.h>

#include "pa_beam.h"
#include "pa_common.cuh"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarpsPerCta = kThreads / 32;
constexpr int kCluster = 8;  // the portable size
constexpr int kSeg = 256;    // table entries of one piece: 8 per lane
// counts below this are claims: INT_MIN + the place of a released entry
constexpr int kClaim = -(1 << 30);

// ---- what both calls share -------------------------------------------------------
struct Pool {
  const int32_t* extra_refs;
  int32_t* extra_refs_out;
  int64_t num_blocks;
  int32_t* free_blocks;
  int64_t free_capacity;
  const int32_t* free_count;
  int32_t* free_count_out;
  unsigned* err;
};

struct Cta {
  int rank, ranks, tid, lane, warp;  // this CTA in the cluster, this thread in it
  int64_t gwarp, gwarps;             // this warp among the cluster's
};
__device__ __forceinline__ Cta this_cta() {
  cg::cluster_group cl = cg::this_cluster();
  Cta t;
  t.rank = (int)cl.block_rank();
  t.ranks = (int)cl.num_blocks();
  t.tid = threadIdx.x;
  t.lane = t.tid & 31;
  t.warp = t.tid >> 5;
  t.gwarp = (int64_t)t.warp * t.ranks + t.rank;
  t.gwarps = (int64_t)kWarpsPerCta * t.ranks;
  return t;
}
// cluster barrier; global writes before it are seen after it
__device__ __forceinline__ void cluster_sync() {
  __threadfence();
  cg::this_cluster().sync();
}

__device__ __forceinline__ void copy_refs(const Pool& p, const Cta& t) {
  if (p.extra_refs == p.extra_refs_out) return;
  const int64_t step = (int64_t)kThreads * t.ranks;
  const int64_t first = (int64_t)t.rank * kThreads + t.tid;
  if (((reinterpret_cast<uintptr_t>(p.extra_refs) |
        reinterpret_cast<uintptr_t>(p.extra_refs_out)) & 15) == 0) {
    const int64_t n4 = p.num_blocks / 4;
    const int4* in = reinterpret_cast<const int4*>(p.extra_refs);
    int4* out = reinterpret_cast<int4*>(p.extra_refs_out);
    for (int64_t i = first; i < n4; i += step) out[i] = in[i];
    for (int64_t i = 4 * n4 + first; i < p.num_blocks; i += step)
      p.extra_refs_out[i] = p.extra_refs[i];
    return;
  }
  for (int64_t i = first; i < p.num_blocks; i += step) p.extra_refs_out[i] = p.extra_refs[i];
}

// The stack's height, 0 with a flag where it is not one.
__device__ __forceinline__ int64_t stack_height(const Pool& p, bool lead) {
  int64_t n = *p.free_count;
  if (n < 0 || n > p.free_capacity) {
    if (lead) flag_error(p.err, PA_DEV_ERR_METADATA);
    n = 0;
  }
  return n;
}

__device__ __forceinline__ bool in_pool(const Pool& p, int id) {
  return id >= 0 && (int64_t)id < p.num_blocks;
}

// The released pieces: piece i is entries [col0, col0 + kSeg) of a row; entry(row,
// col) says whether the call releases it and which block it names.  counts: one
// int per piece, global (pieces <= max_pieces of the plan).
//
// claim(): every released entry of a block out of references proposes itself.
template <class Entry>
__device__ __forceinline__ void claim_released(const Pool& p, const Cta& t, int pieces,
                                               int pieces_per_row, int width,
                                               const Entry& entry) {
  for (int64_t i = t.gwarp; i < pieces; i += t.gwarps) {
    const int k = (int)(i / pieces_per_row), col0 = (int)(i % pieces_per_row) * kSeg;
#pragma unroll
    for (int e = 0; e < kSeg / 32; ++e) {
      int row, id;
      const int col = col0 + e * 32 + t.lane;
      if (!entry(k, col, &row, &id)) continue;
      const int v = __ldcg(p.extra_refs_out + id);
      if (v >= 0) continue;
      if (v < -1 && v > kClaim) flag_error(p.err, PA_DEV_ERR_METADATA);
      atomicMin(p.extra_refs_out + id, INT_MIN + row * width + col);
    }
  }
}
// owners among a piece's entries: a mask per 32 entries
template <class Entry>
__device__ __forceinline__ void owners_of(const Pool& p, const Cta& t, int k, int col0,
                                          int width, const Entry& entry,
                                          unsigned (&mask)[kSeg / 32], int (&ids)[kSeg / 32]) {
  bool mine[kSeg / 32];
#pragma unroll
  for (int e = 0; e < kSeg / 32; ++e) {
    int row;
    const int col = col0 + e * 32 + t.lane;
    mine[e] = entry(k, col, &row, &ids[e]) &&
              __ldcg(p.extra_refs_out + ids[e]) == INT_MIN + row * width + col;
  }
#pragma unroll
  for (int e = 0; e < kSeg / 32; ++e) mask[e] = __ballot_sync(~0u, mine[e]);
}
template <class Entry>
__device__ __forceinline__ void count_owners(const Pool& p, const Cta& t, int pieces,
                                             int pieces_per_row, int width,
                                             const Entry& entry, int* counts) {
  for (int64_t i = t.gwarp; i < pieces; i += t.gwarps) {
    unsigned mask[kSeg / 32];
    int ids[kSeg / 32];
    owners_of(p, t, (int)(i / pieces_per_row), (int)(i % pieces_per_row) * kSeg, width, entry,
              mask, ids);
    int n = 0;
#pragma unroll
    for (int e = 0; e < kSeg / 32; ++e) n += __popc(mask[e]);
    if (t.lane == 0) counts[i] = n;
  }
}
// Pushes the freed blocks from stack position `base` on; returns how many there
// are (in every thread).  scratch: a long long of shared memory and a warp's 32.
template <class Entry>
__device__ __forceinline__ int64_t push_owners(const Pool& p, const Cta& t, int pieces,
                                               int pieces_per_row, int width,
                                               const Entry& entry, const int* counts,
                                               int64_t base, long long* total,
                                               long long* warp_sums, int* starts) {
  // every CTA scans all counts, a round of kThreads at a time, and pushes what its
  // warps have of the round
  int64_t sum = 0;
  for (int first = 0; first < pieces; first += kThreads) {
    const int i = first + t.tid;
    const long long n = i < pieces ? __ldcg(counts + i) : 0;
    const long long before = block_scan_excl(n, total, warp_sums);
    starts[t.tid] = n ? (int)before : -1;
    const int64_t round = *total;
    __syncthreads();
    for (int j = t.warp * t.ranks + t.rank; j < kThreads; j += kWarpsPerCta * t.ranks) {
      const int start = starts[j];
      if (start < 0) continue;  // (same for the whole warp)
      const int piece = first + j;
      unsigned mask[kSeg / 32];
      int ids[kSeg / 32];
      owners_of(p, t, piece / pieces_per_row, piece % pieces_per_row * kSeg, width, entry,
                mask, ids);
      int64_t at = base + sum + start;
#pragma unroll
      for (int e = 0; e < kSeg / 32; ++e) {
        if (mask[e] >> t.lane & 1) {
          const int64_t pos = at + __popc(mask[e] & ((1u << t.lane) - 1));
          if (pos < p.free_capacity)
            p.free_blocks[pos] = ids[e];
          else
            flag_error(p.err, PA_DEV_ERR_METADATA);
          p.extra_refs_out[ids[e]] = 0;
        }
        at += __popc(mask[e]);
      }
    }
    sum += round;
    __syncthreads();  // starts and total are written again
  }
  return sum;
}

// ---- fork --------------------------------------------------------------------------
struct ForkK {
  const int32_t* sources;
  int num_rows;
  const int32_t* tables;
  int32_t* tables_out;
  int width;  // max_blocks_per_seq
  const int32_t* seq_lens;
  int32_t* seq_lens_out;
  Pool pool;
  int64_t* block_mapping;
  int32_t* num_pairs;
  // workspace
  int32_t* row_info;  // [rows] source row, -1: none, or its own in place: nothing to do
  int32_t* row_len;   // [rows] length of the new row
  int32_t* row_last;  // [rows] fresh last block, -1: the source's
  int32_t* row_need;  // [rows] partly filled shared last block (its id), -1: none
  int32_t* counts;    // [pieces]
};

__global__ void __launch_bounds__(kThreads) fork_plan_kernel(ForkK p) {
  extern __shared__ int sh[];
  const int R = p.num_rows;
  int* s_src = sh;            // source of each new row (-1: none)
  int* s_uses = sh + R;       // new rows of each old row
  int* s_len = sh + 2 * R;    // old rows' lengths
  int* s_part = sh + 3 * R;   // new rows' partly filled last block, -1: none
  int* s_gone = sh + 4 * R;   // old rows nobody takes over, in order
  __shared__ int starts[kThreads];
  __shared__ long long warp_sums[32];
  __shared__ long long total;
  const Cta t = this_cta();
  const bool lead = t.rank == 0;
  const Pool& q = p.pool;
  copy_refs(q, t);
  const int64_t height = stack_height(q, lead && t.tid == 0);
  unsigned bad = 0;
  for (int r = t.tid; r < R; r += kThreads) {
    const int s = p.sources[r];
    const int64_t L = p.seq_lens[r];
    const bool fits = L >= 0 && L <= (int64_t)p.width * kBS;
    if (s < -1 || s >= R || !fits) bad = PA_DEV_ERR_METADATA;
    s_src[r] = s < -1 || s >= R ? r : s;
    s_len[r] = fits ? (int)L : 0;
    s_uses[r] = 0;
  }
  if (lead && bad) flag_error(q.err, bad);
  __syncthreads();
  for (int r = t.tid; r < R; r += kThreads)
    if (s_src[r] >= 0) atomicAdd(&s_uses[s_src[r]], 1);
  // sources, lengths and counts are read: the outputs may replace them
  cluster_sync();
  // rows nobody takes over, in order
  int gone = 0;
  for (int base = 0; base < R; base += kThreads) {
    const int r = base + t.tid;
    const bool g = r < R && s_uses[r] == 0;
    const int at = (int)block_scan_excl((long long)g, &total, warp_sums);
    if (g) s_gone[gone + at] = r;
    gone += (int)total;
    __syncthreads();
  }
  // ---- references: u - 1 for each block of an old row that u new rows take over
  const int segs = (p.width + kSeg - 1) / kSeg;
  for (int64_t i = t.gwarp; i < (int64_t)R * segs; i += t.gwarps) {
    const int s = (int)(i / segs), col0 = (int)(i % segs) * kSeg;
    const int change = s_uses[s] - 1;
    const int nb = (s_len[s] + kBS - 1) / kBS;
    if (change == 0 || col0 >= nb) continue;
    const int32_t* row = p.tables + (int64_t)s * p.width;
#pragma unroll
    for (int e = 0; e < kSeg / 32; ++e) {
      const int col = col0 + e * 32 + t.lane;
      if (col >= nb) break;
      const int id = __ldg(row + col);
      if (in_pool(q, id))
        atomicAdd(q.extra_refs_out + id, change);
      else
        flag_error(q.err, PA_DEV_ERR_BLOCK_ID);
    }
  }
  // ---- the new rows' partly filled last blocks (by every CTA for itself)
  for (int r = t.tid; r < R; r += kThreads) {
    const int s = s_src[r];
    int id = -1;
    if (s >= 0 && s_len[s] % kBS != 0) {
      id = __ldg(p.tables + (int64_t)s * p.width + s_len[s] / kBS);
      if (!in_pool(q, id)) {
        flag_error(q.err, PA_DEV_ERR_BLOCK_ID);
        id = -1;
      }
    }
    s_part[r] = id;
  }
  cluster_sync();
  auto entry = [&](int k, int col, int* row, int* id) {
    const int s = s_gone[k];
    *row = s;
    if (col >= (s_len[s] + kBS - 1) / kBS) return false;
    *id = __ldg(p.tables + (int64_t)s * p.width + col);
    return in_pool(q, *id);
  };
  const int pieces = gone * segs;
  claim_released(q, t, pieces, segs, p.width, entry);
  // ---- which rows need a copy of their last block: all that hold it but the first,
  // and that one too where others outside hold it (a warp per row)
  for (int64_t r = t.gwarp; r < R; r += t.gwarps) {
    const int id = s_part[r];
    int need = -1;
    if (id >= 0) {
      int holders = 0, before = 0;
      for (int o = t.lane; o < R; o += 32)
        if (s_part[o] == id) {
          ++holders;
          before += o < r;
        }
      holders = __reduce_add_sync(~0u, holders);
      before = __reduce_add_sync(~0u, before);
      const int others = max(__ldcg(q.extra_refs_out + id), 0) + 1 - holders;
      if (before > 0 || others > 0) need = id;
    }
    if (t.lane == 0) p.row_need[r] = need;
  }
  cluster_sync();
  count_owners(q, t, pieces, segs, p.width, entry, p.counts);
  cluster_sync();
  const int64_t freed = push_owners(q, t, pieces, segs, p.width, entry, p.counts, height,
                                    &total, warp_sums, starts);
  cluster_sync();
  // ---- copies, in row order, onto blocks popped from the stack (the first CTA)
  if (!lead) return;
  const int64_t top = min(height + freed, q.free_capacity);
  int64_t pairs = 0;
  for (int base = 0; base < R; base += kThreads) {
    const int r = base + t.tid;
    const int id = r < R ? __ldcg(p.row_need + r) : -1;
    const int64_t k = pairs + block_scan_excl((long long)(id >= 0), &total, warp_sums);
    int fresh = -1;
    if (id >= 0) {
      if (k < top) {
        fresh = __ldcg(q.free_blocks + (top - 1 - k));
        p.block_mapping[2 * k] = id;
        p.block_mapping[2 * k + 1] = fresh;
        atomicAdd(q.extra_refs_out + id, -1);
        if (!in_pool(q, fresh)) flag_error(q.err, PA_DEV_ERR_BLOCK_ID);
      } else {
        flag_error(q.err, PA_DEV_ERR_NO_BLOCKS);
      }
    }
    if (r < R) {
      const int s = s_src[r];
      const int L = s >= 0 ? s_len[s] : 0;
      p.row_info[r] = s;
      p.row_len[r] = L;
      p.row_last[r] = fresh;
      p.seq_lens_out[r] = L;
    }
    pairs += total;
    __syncthreads();
  }
  pairs = min(pairs, top);
  if (t.tid == 0) {
    *p.num_pairs = (int)pairs;
    *q.free_count_out = (int)(top - pairs);
  }
  for (int64_t k = pairs + t.tid; k < R; k += kThreads)
    p.block_mapping[2 * k] = p.block_mapping[2 * k + 1] = -1;
}

// The new tables.  A CTA takes some columns of all rows: what it will write is read
// first, so that the tables may be changed in place whatever rows trade places.
__global__ void __launch_bounds__(256) fork_tables_kernel(ForkK p, int cols) {
  extern __shared__ int sh[];  // [rows][cols]
  const int col0 = blockIdx.x * cols;
  const bool in_place = p.tables == p.tables_out;
  const int n = p.num_rows * cols;
  pdl_wait();
  for (int i = threadIdx.x; i < n; i += 256) {
    const int r = i / cols, col = col0 + i % cols;
    const int L = __ldcg(p.row_len + r);
    if (col >= (L + kBS - 1) / kBS) continue;
    const int s = __ldcg(p.row_info + r), last = __ldcg(p.row_last + r);
    sh[i] = last != -1 && col == L / kBS ? last : p.tables[(int64_t)s * p.width + col];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 256) {
    const int r = i / cols, col = col0 + i % cols;
    const int L = __ldcg(p.row_len + r);
    if (col >= (L + kBS - 1) / kBS) continue;
    if (in_place && __ldcg(p.row_info + r) == r && __ldcg(p.row_last + r) == -1) continue;
    p.tables_out[(int64_t)r * p.width + col] = sh[i];
  }
}

// ---- compact -----------------------------------------------------------------------
struct CompactK {
  const int32_t* keep;
  int max_keep;
  const int32_t* keep_lens;
  const int32_t* keep_start;
  int num_rows;
  const int32_t* tables;
  int32_t* tables_out;
  int width;
  const int32_t* seq_lens;
  int32_t* seq_lens_out;
  Pool pool;
  int64_t* src_slots;
  int64_t* dst_slots;
  int32_t* num_moves;
  // workspace
  int32_t* same;    // [rows] listed tokens that stay where they are
  int32_t* broken;  // [rows] the list is not one
  int32_t* info;    // [rows][4]: tokens kept (-1: as it is), first changed block, old
                    // length, moves
  int32_t* fresh;   // [rows][width], of the changed blocks: the id that replaces it,
                    // INT_MIN: none does
  int32_t* counts;  // [pieces]
  int32_t* bases;   // [pieces] blocks popped before a piece's
};

__global__ void __launch_bounds__(kThreads) compact_plan_kernel(CompactK p) {
  extern __shared__ int sh[];
  const int R = p.num_rows;
  int* s_len = sh;            // old lengths
  int* s_n = sh + R;          // tokens kept (-1: the row stays as it is)
  int* s_first = sh + 2 * R;  // first block that changes
  int* s_end = sh + 3 * R;    // blocks popped up to and including the row
  __shared__ int starts[kThreads];
  __shared__ long long warp_sums[32];
  __shared__ long long total;
  __shared__ int s_popped;
  const Cta t = this_cta();
  const bool lead = t.rank == 0;
  const Pool& q = p.pool;
  copy_refs(q, t);
  const int64_t height = stack_height(q, lead && t.tid == 0);
  unsigned bad = 0;
  for (int r = t.tid; r < R; r += kThreads) {
    const int64_t L = p.seq_lens[r];
    const int k = p.keep_lens[r], start = p.keep_start ? p.keep_start[r] : 0;
    const bool fits = L >= 0 && L <= (int64_t)p.width * kBS;
    const bool ok = fits && k <= p.max_keep && (k < 0 || (start >= 0 && start <= L));
    if (!ok) bad = PA_DEV_ERR_METADATA;
    s_len[r] = fits ? (int)L : 0;
    s_n[r] = ok && k >= 0 ? start + k : -1;
    s_first[r] = start;
    if (lead) p.same[r] = p.broken[r] = 0;
  }
  if (lead && bad) flag_error(q.err, bad);
  if (t.tid == 0) s_popped = 0;
  cluster_sync();
  // ---- the lists: ascending positions in [start, L); how many stay in place
  const int lsegs = (p.max_keep + kSeg - 1) / kSeg;
  for (int64_t i = t.gwarp; i < (int64_t)R * lsegs; i += t.gwarps) {
    const int r = (int)(i / lsegs), j0 = (int)(i % lsegs) * kSeg;
    const int start = s_first[r], k = s_n[r] - start;
    if (s_n[r] < 0 || j0 >= k) continue;
    const int32_t* list = p.keep + (int64_t)r * p.max_keep;
    int same = 0;
    bool ok = true;
#pragma unroll
    for (int e = 0; e < kSeg / 32; ++e) {
      const int j = j0 + e * 32 + t.lane;
      if (j >= k) break;
      const int v = __ldg(list + j);
      const int before = j ? __ldg(list + j - 1) : start - 1;
      ok = ok && v > before && v < s_len[r];
      same += v == start + j;
    }
    same = __reduce_add_sync(~0u, same);
    const bool all = __all_sync(~0u, ok);
    if (t.lane == 0) {
      if (same) atomicAdd(p.same + r, same);
      if (!all) p.broken[r] = 1;
    }
  }
  cluster_sync();
  bad = 0;
  for (int r = t.tid; r < R; r += kThreads) {
    if (s_n[r] < 0) continue;
    if (__ldcg(p.broken + r)) {
      bad = PA_DEV_ERR_METADATA;
      s_n[r] = -1;
    } else {
      s_first[r] = (s_first[r] + __ldcg(p.same + r)) / kBS;
    }
  }
  if (lead && bad) flag_error(q.err, bad);
  __syncthreads();
  // ---- blocks that change and have other holders: replaced by fresh ones
  const int segs = (p.width + kSeg - 1) / kSeg;
  const int pieces = R * segs;
  auto shared_of = [&](int r, int col0, unsigned (&mask)[kSeg / 32]) {
    const int left = (s_n[r] + kBS - 1) / kBS;
    const int32_t* row = p.tables + (int64_t)r * p.width;
    bool shared[kSeg / 32];
#pragma unroll
    for (int e = 0; e < kSeg / 32; ++e) {
      const int col = col0 + e * 32 + t.lane;
      shared[e] = false;
      if (col >= s_first[r] && col < left) {
        const int id = __ldg(row + col);
        shared[e] = in_pool(q, id) && __ldcg(q.extra_refs + id) > 0;
      }
    }
#pragma unroll
    for (int e = 0; e < kSeg / 32; ++e) mask[e] = __ballot_sync(~0u, shared[e]);
  };
  auto changes = [&](int r, int col0) {  // any block of a piece that may change
    return s_n[r] > col0 * kBS && col0 + kSeg > s_first[r];
  };
  for (int64_t i = t.gwarp; i < pieces; i += t.gwarps) {
    const int r = (int)(i / segs), col0 = (int)(i % segs) * kSeg;
    int n = 0;
    if (changes(r, col0)) {
      unsigned mask[kSeg / 32];
      shared_of(r, col0, mask);
#pragma unroll
      for (int e = 0; e < kSeg / 32; ++e) n += __popc(mask[e]);
    }
    if (t.lane == 0) p.counts[i] = n;
  }
  cluster_sync();
  // ---- pops in row order; the rows whose running need fits the stack run
  int64_t sum = 0;
  for (int base = 0; base < pieces; base += kThreads) {
    const int i = base + t.tid;
    const long long n = i < pieces ? __ldcg(p.counts + i) : 0;
    const int64_t before = sum + block_scan_excl(n, &total, warp_sums);
    if (i < pieces) {
      if (lead) p.bases[i] = (int)before;
      if (i % segs == segs - 1) s_end[i / segs] = (int)(before + n);
    }
    sum += total;
    __syncthreads();
  }
  cluster_sync();
  bad = 0;
  for (int r = t.tid; r < R; r += kThreads) {
    if (pieces > 0 && s_end[r] > height) {
      bad = PA_DEV_ERR_NO_BLOCKS;
      s_n[r] = -1;
    } else if (pieces > 0) {
      atomicMax(&s_popped, s_end[r]);
    }
  }
  if (lead && bad) flag_error(q.err, bad);
  __syncthreads();
  const int64_t popped = s_popped;
  // ---- fresh ids.  What is shared is told by the counts before any of them changes,
  // and is marked in p.fresh for what follows.
  for (int64_t i = t.gwarp; i < pieces; i += t.gwarps) {
    const int r = (int)(i / segs), col0 = (int)(i % segs) * kSeg;
    if (!changes(r, col0)) continue;
    const int left = (s_n[r] + kBS - 1) / kBS;
    unsigned mask[kSeg / 32];
    shared_of(r, col0, mask);
    int64_t nth = __ldcg(p.bases + i);
#pragma unroll
    for (int e = 0; e < kSeg / 32; ++e) {
      const int col = col0 + e * 32 + t.lane;
      if (col >= s_first[r] && col < left) {
        int fresh = INT_MIN;
        if (mask[e] >> t.lane & 1) {
          fresh = __ldcg(q.free_blocks +
                         (height - 1 - nth - __popc(mask[e] & ((1u << t.lane) - 1))));
          if (!in_pool(q, fresh)) {
            flag_error(q.err, PA_DEV_ERR_BLOCK_ID);
            fresh = -1;
          }
        }
        p.fresh[(int64_t)r * p.width + col] = fresh;
      }
      nth += __popc(mask[e]);
    }
  }
  cluster_sync();
  auto entry = [&](int r, int col, int* row, int* id) {
    *row = r;
    const int n = s_n[r];
    if (n < 0 || col < s_first[r] || col >= (s_len[r] + kBS - 1) / kBS) return false;
    if (col < (n + kBS - 1) / kBS && __ldcg(p.fresh + (int64_t)r * p.width + col) == INT_MIN)
      return false;
    *id = __ldg(p.tables + (int64_t)r * p.width + col);
    return in_pool(q, *id);
  };
  for (int64_t i = t.gwarp; i < pieces; i += t.gwarps) {
    const int r = (int)(i / segs), col0 = (int)(i % segs) * kSeg;
#pragma unroll
    for (int e = 0; e < kSeg / 32; ++e) {
      int row, id;
      if (entry(r, col0 + e * 32 + t.lane, &row, &id)) atomicAdd(q.extra_refs_out + id, -1);
    }
  }
  cluster_sync();
  claim_released(q, t, pieces, segs, p.width, entry);
  cluster_sync();
  count_owners(q, t, pieces, segs, p.width, entry, p.counts);
  cluster_sync();
  // the popped ids are read: pushes may take their places
  const int64_t freed = push_owners(q, t, pieces, segs, p.width, entry, p.counts,
                                    height - popped, &total, warp_sums, starts);
  if (!lead) return;
  if (t.tid == 0)
    *q.free_count_out = (int)min(height - popped + freed, q.free_capacity);
  for (int r = t.tid; r < R; r += kThreads) {
    const int n = s_n[r], first = s_first[r];
    int moves = 0;
    if (n >= 0) {
      // a row that only loses its end moves nothing, unless its last block is replaced
      const int start = p.keep_start ? p.keep_start[r] : 0;
      const bool whole = start + __ldcg(p.same + r) == n;
      const bool swapped = first * kBS < n &&
                           __ldcg(p.fresh + (int64_t)r * p.width + first) != INT_MIN;
      if (!whole || swapped) moves = n - first * kBS;
    }
    p.num_moves[r] = moves;
    int4 info = make_int4(n, first, s_len[r], moves);
    reinterpret_cast<int4*>(p.info)[r] = info;
    p.seq_lens_out[r] = n >= 0 ? n : s_len[r];
  }
}

// The moves: a thread per listed place.
__global__ void __launch_bounds__(256) compact_moves_kernel(CompactK p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t wide = p.max_keep + kBS;
  const int r = blockIdx.y;
  const int4 info = __ldcg(reinterpret_cast<const int4*>(p.info) + r);
  const int32_t* row = p.tables + (int64_t)r * p.width;
  const int32_t* fresh = p.fresh + (int64_t)r * p.width;
  const int start = info.w ? (p.keep_start ? p.keep_start[r] : 0) : 0;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < info.w; i += gridDim.x * 256) {
    const int at = info.y * kBS + i;
    const int pos = at < start ? at : p.keep[(int64_t)r * p.max_keep + at - start];
    const int from = row[pos / kBS];
    const int was = row[at / kBS], now = fresh[at / kBS];
    const int to = now == INT_MIN ? was : now;
    const bool ok = from >= 0 && from < p.pool.num_blocks && to >= 0 &&
                    to < p.pool.num_blocks;
    if (!ok) flag_error(p.pool.err, PA_DEV_ERR_BLOCK_ID);
    p.src_slots[r * wide + i] = ok ? (int64_t)from * kBS + pos % kBS : -1;
    p.dst_slots[r * wide + i] = ok ? (int64_t)to * kBS + at % kBS : -1;
  }
}

// The tables: in place, only what is replaced.
__global__ void __launch_bounds__(256) compact_tables_kernel(CompactK p) {
  pdl_wait();
  const int r = blockIdx.y;
  const int4 info = __ldcg(reinterpret_cast<const int4*>(p.info) + r);
  const bool in_place = p.tables == p.tables_out;
  const int blocks = ((info.x >= 0 ? info.x : info.z) + kBS - 1) / kBS;
  const int64_t at = (int64_t)r * p.width;
  for (int col = blockIdx.x * 256 + threadIdx.x; col < blocks; col += gridDim.x * 256) {
    const int now = info.x >= 0 && col >= info.y ? p.fresh[at + col] : INT_MIN;
    if (now != INT_MIN)
      p.tables_out[at + col] = now;
    else if (!in_place)
      p.tables_out[at + col] = p.tables[at + col];
  }
}

template <class P>
cudaError_t launch_plan(void (*kernel)(P), const P& p, size_t smem, size_t max_smem,
                        cudaStream_t stream) {
  // (always the largest step's limit: see launch_build_step)
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)max_smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kCluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <class... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, size_t smem, cudaStream_t stream,
                         A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e == cudaSuccess) count_launch();
  return e;
}

Pool pool_of(const RowState& r, unsigned* err) {
  return Pool{r.extra_refs,    r.extra_refs_out, r.num_blocks,     r.free_blocks,
              r.free_capacity, r.free_count,     r.free_count_out, err};
}

int64_t pieces_of(int64_t rows, int64_t width) { return rows * ((width + kSeg - 1) / kSeg); }

}  // namespace

int64_t fork_workspace_bytes(int num_rows, int max_blocks_per_seq) {
  return 4 * (4ll * num_rows + pieces_of(num_rows, max_blocks_per_seq));
}

cudaError_t launch_fork_blocks(const ForkArgs& a, cudaStream_t stream) {
  ForkK p{};
  p.sources = a.sources;
  p.num_rows = a.rows.num_rows;
  p.tables = a.rows.block_tables;
  p.tables_out = a.rows.block_tables_out;
  p.width = a.rows.max_blocks_per_seq;
  p.seq_lens = a.rows.seq_lens;
  p.seq_lens_out = a.rows.seq_lens_out;
  p.pool = pool_of(a.rows, a.err);
  p.block_mapping = a.block_mapping;
  p.num_pairs = a.num_pairs;
  const int64_t R = a.rows.num_rows;
  p.row_info = static_cast<int32_t*>(a.workspace);
  p.row_len = p.row_info + R;
  p.row_last = p.row_len + R;
  p.row_need = p.row_last + R;
  p.counts = p.row_need + R;
  cudaError_t e = launch_plan(fork_plan_kernel, p, (size_t)(5 * R * 4),
                              (size_t)5 * kMaxForkRows * 4, stream);
  if (e != cudaSuccess || R == 0 || p.width == 0) return e;
  // columns of a CTA: a line of 32 where all rows' fit 40 KB of shared memory, 2 of
  // them at the largest number of rows
  int cols = 32;
  while ((int64_t)cols * R * 4 > 40 * 1024 && cols > 2) cols /= 2;
  return launch_after(fork_tables_kernel, dim3((unsigned)((p.width + cols - 1) / cols)),
                      (size_t)cols * R * 4, stream, p, cols);
}

int64_t compact_workspace_bytes(int num_rows, int max_blocks_per_seq) {
  return 4 * (6ll * num_rows + (int64_t)num_rows * max_blocks_per_seq +
              2 * pieces_of(num_rows, max_blocks_per_seq));
}

cudaError_t launch_compact_blocks(const CompactArgs& a, cudaStream_t stream) {
  CompactK p{};
  p.keep = a.keep;
  p.max_keep = a.max_keep;
  p.keep_lens = a.keep_lens;
  p.keep_start = a.keep_start;
  p.num_rows = a.rows.num_rows;
  p.tables = a.rows.block_tables;
  p.tables_out = a.rows.block_tables_out;
  p.width = a.rows.max_blocks_per_seq;
  p.seq_lens = a.rows.seq_lens;
  p.seq_lens_out = a.rows.seq_lens_out;
  p.pool = pool_of(a.rows, a.err);
  p.src_slots = a.src_slots;
  p.dst_slots = a.dst_slots;
  p.num_moves = a.num_moves;
  const int64_t R = a.rows.num_rows;
  p.info = static_cast<int32_t*>(a.workspace);  // 16-byte aligned
  p.same = p.info + 4 * R;
  p.broken = p.same + R;
  p.counts = p.broken + R;
  p.bases = p.counts + pieces_of(R, p.width);
  p.fresh = p.bases + pieces_of(R, p.width);
  cudaError_t e = launch_plan(compact_plan_kernel, p, (size_t)(4 * R * 4),
                              (size_t)4 * kMaxForkRows * 4, stream);
  if (e != cudaSuccess || R == 0 || p.width == 0) return e;
  const int64_t wide = (int64_t)p.max_keep + kBS;
  const unsigned gm = (unsigned)((wide + 255) / 256 < 64 ? (wide + 255) / 256 : 64);
  e = launch_after(compact_moves_kernel, dim3(gm, (unsigned)R), 0, stream, p);
  if (e != cudaSuccess) return e;
  const unsigned gt = (unsigned)((p.width + 255) / 256 < 64 ? (p.width + 255) / 256 : 64);
  return launch_after(compact_tables_kernel, dim3(gt, (unsigned)R), 0, stream, p);
}

}  // namespace pa
