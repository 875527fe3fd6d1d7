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
// Shape.  A few MB at most are read and written (tables, counts, lists), but by
// passes that each need all of the one before: references, claims, owners counted,
// owners pushed, tables.  So a call is one kernel whose CTAs meet at a barrier
// between the passes: up to eight or sixteen CTAs as one cluster, where more are needed
// a cooperative grid (one CTA per SM at most).  Every CTA keeps the rows' sources and
// lengths in shared memory and does the small scans over rows or pieces for itself.
// Tables are walked as far as the longest row goes, not as wide as they are.  (They are
// read by ordinary loads: the call may write them, once nobody reads the old ones.)
// What is left is latency: five or six barriers of 1.3 us each, the way of the writes
// before them to L2 included, and one or two loads of 0.5 us between them.  64 forked
// rows of up to 258 blocks 13 us, 1024 of up to 1026 29 us; 64 requests that keep 6
// of their last 32 tokens 15.5 us, 32 prompts of 2K to 32K that keep a quarter 30 us.
#include <cooperative_groups.h>
#include <limits.h>

#include "pa_beam.h"
#include "pa_common.cuh"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarpsPerCta = kThreads / 32;
constexpr int kMaxCluster = 8;   // the portable size
constexpr int kBigCluster = 16;  // where the device can hold it
constexpr int kSeg = 256;       // table entries (or listed tokens) of one piece: 8 per lane
constexpr int kPer = kSeg / 32;
constexpr int kFewPieces = 8;   // that every CTA of a cluster looks through for itself
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

// The CTAs of a call, and this thread's place among them.
struct Team {
  int rank, ranks, tid, lane, warp;
  int gwarp, gwarps;  // this warp among all
  bool cluster;
  __device__ __forceinline__ explicit Team(bool one_cluster) : cluster(one_cluster) {
    rank = (int)blockIdx.x;
    ranks = (int)gridDim.x;
    tid = threadIdx.x;
    lane = tid & 31;
    warp = tid >> 5;
    gwarp = warp * ranks + rank;
    gwarps = kWarpsPerCta * ranks;
  }
  // global writes before it are seen after it, by all
  __device__ __forceinline__ void sync() const {
    if (cluster) {
      cg::this_cluster().sync();  // (a release and an acquire of global writes, too)
    } else {
      cg::this_grid().sync();
    }
  }
};

__device__ __forceinline__ void copy_refs(const Pool& p, const Team& t) {
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

// The stack's height as it was read, 0 with a flag where it is not one.
__device__ __forceinline__ int64_t stack_height(const Pool& p, int64_t n, bool lead) {
  if (n < 0 || n > p.free_capacity) {
    if (lead) flag_error(p.err, PA_DEV_ERR_METADATA);
    n = 0;
  }
  return n;
}

__device__ __forceinline__ bool in_pool(const Pool& p, int id) {
  return id >= 0 && (int64_t)id < p.num_blocks;
}

// Counts of one round of a scan: one to a thread, or four where there are more pieces than
// threads (1024 rows of up to 1026 blocks, some 2500 released pieces: 31.0 us with one, 29.2
// with four; 64 rows of up to 258, some 30 pieces: 14.2 and 14.4 then).
constexpr int kEach = 4, kScan = kEach * kThreads;

struct Scan {  // shared memory of the scans
  int warp_sums[32];
  int total;
  int starts[kScan];
};

// The CTA's largest v, after the barrier that follows put().
struct Largest {
  int* room;  // [32]
  __device__ __forceinline__ void put(const Team& t, int v) const {
    v = __reduce_max_sync(~0u, v);
    if (t.lane == 0) room[t.warp] = v;
  }
  __device__ __forceinline__ int get(const Team& t) const {
    return __reduce_max_sync(~0u, room[t.lane]);
  }
};

// f(piece, sum of the counts before it) for each piece whose count is not 0, by the
// warp that it belongs to; the sum of all counts, in every thread.
template <class F>
__device__ __forceinline__ int64_t in_order(const Team& t, int pieces, const int* counts,
                                            Scan& sh, const F& f) {
  int64_t sum = 0;
  const int each = pieces > kThreads ? kEach : 1;
#pragma unroll 1
  for (int first = 0; first < pieces; first += each * kThreads) {
    int n[kEach], mine = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = first + t.tid * each + e;
      n[e] = e < each && i < pieces ? __ldcg(counts + i) : 0;
      mine += n[e];
    }
    int before = block_scan_excl(mine, &sh.total, sh.warp_sums);
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (e < each) {
        sh.starts[t.tid * each + e] = n[e] ? before : -1;
        before += n[e];
      }
    const int64_t round = sh.total;
    __syncthreads();
    const int ahead = first % t.gwarps, here = min(each * kThreads, pieces - first);
#pragma unroll 1
    for (int j = t.gwarp >= ahead ? t.gwarp - ahead : t.gwarp - ahead + t.gwarps; j < here;
         j += t.gwarps)
      if (sh.starts[j] >= 0) f(first + j, sum + sh.starts[j]);
    sum += round;
    __syncthreads();  // starts and total are written again
  }
  return sum;
}

// The entries that a call releases, in pieces: piece i is entries [col0, col0 + kSeg) of
// the (i / per_row)-th row that releases any.  load(k, col0, ids): the blocks that the
// released entries among them name, -1 elsewhere (entry e of a lane: column col0 + 32 e +
// lane; any number in a broken table); row_of(k): the row.  A piece belongs to the same warp
// in every pass, which keeps its first piece's blocks and, once known, owners in registers:
// most calls have no more pieces than warps, and then a pass is one load of the counts.
template <class Load, class RowOf>
struct Released {
  const Pool& p;
  const Team& t;
  const int me, all;  // this warp among those that share the pieces
  const int pieces, per_row, width;
  const Load& load;
  const RowOf& row_of;
  int first_ids[kPer], first_counts[kPer];
  unsigned first_owners[kPer];

  __device__ __forceinline__ Released(const Pool& pool, const Team& team, bool alone,
                                      int n_pieces, int pieces_per_row, int table_width,
                                      const Load& l, const RowOf& r)
      : p(pool), t(team), me(alone ? team.warp : team.gwarp),
        all(alone ? kWarpsPerCta : team.gwarps), pieces(n_pieces), per_row(pieces_per_row),
        width(table_width), load(l), row_of(r) {
    if (me < pieces) fetch(me, first_ids);
  }
  // the first piece's counts, loaded ahead of claim() or count()
  __device__ __forceinline__ void look_ahead() {
    if (me < pieces) counts_of(first_ids, first_counts);
  }
  // every released entry of a block out of references proposes itself
  __device__ __forceinline__ void claim() const {
#pragma unroll 1
    for (int i = me; i < pieces; i += all) {
      int ids[kPer], count[kPer];
      get(i, ids, count);
      const int at = place(i);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (count[e] >= 0) continue;
        if (count[e] < -1 && count[e] > kClaim) flag_error(p.err, PA_DEV_ERR_METADATA);
        atomicMin(p.extra_refs_out + ids[e], at + 32 * e);
      }
    }
  }
  // the blocks that each piece owns, into counts
  __device__ __forceinline__ void count(int* counts) {
#pragma unroll 1
    for (int i = me; i < pieces; i += all) {
      int ids[kPer], count[kPer], n = 0;
      unsigned owners[kPer];
      get(i, ids, count);
      owners_of(i, count, owners);
#pragma unroll
      for (int e = 0; e < kPer; ++e) n += __popc(owners[e]);
      if (i == me)
#pragma unroll
        for (int e = 0; e < kPer; ++e) first_owners[e] = owners[e];
      if (t.lane == 0) counts[i] = n;
    }
  }
  // Where every CTA has all pieces, one to a warp at most: how many blocks this one owns,
  // and f(which of them, block) for each.
  __device__ __forceinline__ int own() {
    int n = 0;
    if (me < pieces) {
      owners_of(me, first_counts, first_owners);
#pragma unroll
      for (int e = 0; e < kPer; ++e) n += __popc(first_owners[e]);
    }
    return n;
  }
  template <class F>
  __device__ __forceinline__ void each_owned(const F& f) const {
    if (me >= pieces) return;
    int at = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      if (first_owners[e] >> t.lane & 1)
        f(at + __popc(first_owners[e] & ((1u << t.lane) - 1)), first_ids[e]);
      at += __popc(first_owners[e]);
    }
  }
  // Pushes them from stack position `base` on; how many there are.  (Every CTA scans all
  // counts.)
  __device__ __forceinline__ int64_t push(const int* counts, int64_t base, Scan& sh) const {
    return in_order(t, pieces, counts, sh, [&](int i, int64_t before) {
      int ids[kPer], count[kPer];
      unsigned owners[kPer];
      if (i == me) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          ids[e] = first_ids[e];
          owners[e] = first_owners[e];
        }
      } else {
        get(i, ids, count);
        owners_of(i, count, owners);
      }
      int64_t at = base + before;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (owners[e] >> t.lane & 1) {
          const int64_t pos = at + __popc(owners[e] & ((1u << t.lane) - 1));
          if (pos < p.free_capacity)
            p.free_blocks[pos] = ids[e];
          else
            flag_error(p.err, PA_DEV_ERR_METADATA);
          p.extra_refs_out[ids[e]] = 0;
        }
        at += __popc(owners[e]);
      }
    });
  }

 private:
  __device__ __forceinline__ void fetch(int i, int (&ids)[kPer]) const {
    load(i / per_row, i % per_row * kSeg, ids);
  }
  // the claim of a piece's entry 0 of this lane
  __device__ __forceinline__ int place(int i) const {
    return INT_MIN + row_of(i / per_row) * width + i % per_row * kSeg + t.lane;
  }
  __device__ __forceinline__ void counts_of(const int (&ids)[kPer], int (&count)[kPer]) const {
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      count[e] = in_pool(p, ids[e]) ? __ldcg(p.extra_refs_out + ids[e]) : 0;
  }
  __device__ __forceinline__ void get(int i, int (&ids)[kPer], int (&count)[kPer]) const {
    if (i == me) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        ids[e] = first_ids[e];
        count[e] = first_counts[e];
      }
    } else {
      fetch(i, ids);
      counts_of(ids, count);
    }
  }
  __device__ __forceinline__ void owners_of(int i, const int (&count)[kPer],
                                            unsigned (&owners)[kPer]) const {
    const int at = place(i);
#pragma unroll
    for (int e = 0; e < kPer; ++e) owners[e] = __ballot_sync(~0u, count[e] == at + 32 * e);
  }
};

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
  int cols_log2;  // table columns of one tile
  bool cluster;
  // workspace
  int32_t* row_need;  // [rows] partly filled shared last block (its id), -1: none
  int32_t* counts;    // [pieces]
};

__global__ void __launch_bounds__(kThreads, 1) fork_kernel(ForkK p) {
  extern __shared__ int sh[];
  const int R = p.num_rows;
  int* s_src = sh;            // source of each new row (-1: none)
  int* s_uses = sh + R;       // new rows of each old row; then each new row's place among
                              // the copies, -1: none; then -1 too where the stack ran out
  int* s_len = sh + 2 * R;    // old rows' lengths
  int* s_part = sh + 3 * R;   // new rows' partly filled last block, -1: none; then that to
                              // be copied; then what was popped in its place (any number)
  int* s_gone = sh + 4 * R;   // old rows nobody takes over, in order
  int* s_tile = sh + 5 * R;   // [rows][cols] of the new tables
  __shared__ Scan scan;
  const Team t(p.cluster);
  const bool lead = t.rank == 0;
  const Pool& q = p.pool;
  const int counted = *q.free_count;
  unsigned bad = 0;
  int longest = 0;
  const Largest of_lengths{scan.starts};
  for (int r = t.tid; r < R; r += kThreads) {
    const int s = __ldg(p.sources + r);
    const int64_t L = p.seq_lens[r];
    const bool fits = L >= 0 && L <= (int64_t)p.width * kBS;
    if (s < -1 || s >= R || !fits) bad = PA_DEV_ERR_METADATA;
    s_src[r] = s < -1 || s >= R ? r : s;
    s_len[r] = fits ? (int)L : 0;
    s_uses[r] = 0;
    longest = max(longest, s_len[r]);
  }
  of_lengths.put(t, longest);
  if (lead && bad) flag_error(q.err, bad);
  __syncthreads();
  const int filled = (of_lengths.get(t) + kBS - 1) / kBS;  // columns of the longest row
  for (int r = t.tid; r < R; r += kThreads)
    if (s_src[r] >= 0) atomicAdd(&s_uses[s_src[r]], 1);
  __syncthreads();
  // ---- the rows nobody takes over, in order
  int gone = 0;
#pragma unroll 1
  for (int base = 0; base < R; base += kThreads) {
    const int r = base + t.tid;
    const bool g = r < R && s_uses[r] == 0 && s_len[r] > 0;
    const int at = block_scan_excl((int)g, &scan.total, scan.warp_sums);
    if (g) s_gone[gone + at] = r;
    gone += scan.total;
    __syncthreads();
  }
  // ---- what needs only the inputs is loaded before the counts are settled, all of it
  // before any of it is looked at: this warp's first pieces of the old rows' tables and of
  // the released ones, and the new rows' partly filled last blocks (by every CTA for itself)
  const int segs = (max(filled, min(p.width, 1)) + kSeg - 1) / kSeg;  // (0: no columns)
  auto entries = [&](int s, int col0, int (&ids)[kPer]) {
    const int nb = (s_len[s] + kBS - 1) / kBS;
    const int32_t* row = p.tables + (int64_t)s * p.width;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int col = col0 + e * 32 + t.lane;
      ids[e] = col < nb ? row[col] : -1;
    }
  };
  int ids[kPer];
  int i = t.gwarp;
  for (; i < R * segs; i += t.gwarps) {
    if (s_uses[i / segs] == 1) continue;
    entries(i / segs, i % segs * kSeg, ids);
    break;
  }
  auto load = [&](int k, int col0, int (&out)[kPer]) { entries(s_gone[k], col0, out); };
  auto row_of = [&](int k) { return s_gone[k]; };
  // Few pieces, and all CTAs in one cluster: every CTA finds and counts the freed blocks for
  // itself, which saves two barriers and the ways to memory between them (4 rows of 63 blocks
  // 13.2 -> 10.9 us; with 23 pieces of 256, 64 rows, it would be 13.9 -> 19.5).
  const bool alone = p.cluster && gone * segs <= kFewPieces;
  Released<decltype(load), decltype(row_of)> released(q, t, alone, gone * segs, segs, p.width,
                                                      load, row_of);
#pragma unroll 1
  for (int r = t.tid; r < R; r += kThreads) {
    const int s = s_src[r];
    int id = -1;
    if (s >= 0 && s_len[s] % kBS != 0) {
      id = p.tables[(int64_t)s * p.width + s_len[s] / kBS];
      if (!in_pool(q, id)) {
        if (lead) flag_error(q.err, PA_DEV_ERR_BLOCK_ID);
        id = -1;
      }
    }
    s_part[r] = id;
  }
  if (q.extra_refs != q.extra_refs_out) {
    copy_refs(q, t);
    t.sync();
  }
  // ---- references: u - 1 for each block of an old row that u new rows take over
#pragma unroll 1
  while (i < R * segs) {
    const int change = s_uses[i / segs] - 1, nb = (s_len[i / segs] + kBS - 1) / kBS;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      if (in_pool(q, ids[e]))
        atomicAdd(q.extra_refs_out + ids[e], change);
      else if (i % segs * kSeg + e * 32 + t.lane < nb)
        flag_error(q.err, PA_DEV_ERR_BLOCK_ID);
    }
    for (i += t.gwarps; i < R * segs; i += t.gwarps) {
      if (s_uses[i / segs] == 1) continue;
      entries(i / segs, i % segs * kSeg, ids);
      break;
    }
  }
  t.sync();
  released.look_ahead();
  // ---- which rows need a copy of their last block: all that hold it but the first,
  // and that one too where others outside hold it (a warp per row)
#pragma unroll 1
  for (int r = t.gwarp; r < R; r += t.gwarps) {
    const int id = s_part[r];
    int need = -1;
    if (id >= 0) {
      const int extra = __ldcg(q.extra_refs_out + id);
      int holders = 0, before = 0;
#pragma unroll 1
      for (int o = t.lane; o < R; o += 32)
        if (s_part[o] == id) {
          ++holders;
          before += o < r;
        }
      holders = __reduce_add_sync(~0u, holders);
      before = __reduce_add_sync(~0u, before);
      if (before > 0 || max(extra, 0) + 1 - holders > 0) need = id;
    }
    if (t.lane == 0) p.row_need[r] = need;
  }
  if (!alone || t.warp % t.ranks == t.rank) released.claim();
  t.sync();
  const int64_t height = stack_height(q, counted, lead && t.tid == 0);
  released.look_ahead();
  // ---- the copies' numbers, while the freed blocks are counted
  int64_t pairs = 0;
#pragma unroll 1
  for (int base = 0; base < R; base += kThreads) {
    const int r = base + t.tid;
    const int id = r < R ? __ldcg(p.row_need + r) : -1;
    const int k = (int)pairs + block_scan_excl((int)(id >= 0), &scan.total, scan.warp_sums);
    if (r < R) {
      s_part[r] = id;
      s_uses[r] = id >= 0 ? k : -1;
    }
    pairs += scan.total;
    __syncthreads();
  }
  // ---- the new tables.  A CTA takes some columns of all rows: what it will write is
  // read first, so that the tables may be changed in place whatever rows trade places.
  // (The first columns now: nobody writes to the tables before the last barrier.)
  const int cols = 1 << p.cols_log2, items = R << p.cols_log2;
  auto read_tile = [&](int col0) {
#pragma unroll 8
    for (int i = t.tid; i < items; i += kThreads) {
      const int r = i >> p.cols_log2, col = col0 + (i & (cols - 1)), s = s_src[r];
      if (s >= 0 && col < (s_len[s] + kBS - 1) / kBS)
        s_tile[i] = p.tables[(int64_t)s * p.width + col];
    }
  };
  if (t.rank * cols < filled) read_tile(t.rank * cols);
  int64_t freed = 0, top;
  int* s_fresh = s_gone;  // the freed blocks among those to be popped, in their order
  if (alone) {            // (the same in every CTA)
    const int mine = released.own();
    if (t.lane == 0) scan.starts[t.warp] = mine;
    cg::this_cluster().barrier_arrive();  // (the claims have been read)
    __syncthreads();
    const int n = scan.starts[t.lane];
    freed = __reduce_add_sync(~0u, n);
    top = min(height + freed, q.free_capacity);
    const int64_t base = height + __reduce_add_sync(~0u, t.lane < t.warp ? n : 0);
    released.each_owned([&](int at, int id) {
      const int64_t pos = base + at;
      if (pos >= q.free_capacity) {
        if (lead) flag_error(q.err, PA_DEV_ERR_METADATA);
        return;
      }
      if (lead) q.free_blocks[pos] = id;
      if (top - 1 - pos < pairs) s_fresh[top - 1 - pos] = id;
    });
    __syncthreads();
  } else {
    if (gone > 0) {
      released.count(p.counts);
      t.sync();
      freed = released.push(p.counts, height, scan);
    }
    t.sync();
    top = min(height + freed, q.free_capacity);
  }
  // ---- copies, in row order, onto blocks popped from the stack
  for (int r = t.tid; r < R; r += kThreads) {
    const int id = s_part[r], k = s_uses[r];
    int fresh = -1;
    if (k >= 0 && k < top) {
      if (alone && top - 1 - k >= height)
        fresh = s_fresh[k];
      else
        fresh = __ldcg(q.free_blocks + (top - 1 - k));
    }
    s_part[r] = fresh;
    if (lead && k >= 0) {
      if (k < top) {
        p.block_mapping[2 * k] = id;
        p.block_mapping[2 * k + 1] = fresh;
        atomicAdd(q.extra_refs_out + id, -1);
        if (!in_pool(q, fresh)) flag_error(q.err, PA_DEV_ERR_BLOCK_ID);
      } else {
        flag_error(q.err, PA_DEV_ERR_NO_BLOCKS);
      }
    }
    if (k >= top) s_uses[r] = -1;
  }
  __syncthreads();
  pairs = min(pairs, top);
  if (lead) {
    if (t.tid == 0) {
      *p.num_pairs = (int)pairs;
      *q.free_count_out = (int)(top - pairs);
    }
    for (int64_t k = pairs + t.tid; k < R; k += kThreads)
      p.block_mapping[2 * k] = p.block_mapping[2 * k + 1] = -1;
    for (int r = t.tid; r < R; r += kThreads)
      p.seq_lens_out[r] = s_src[r] >= 0 ? s_len[s_src[r]] : 0;
  }
  const bool in_place = p.tables == p.tables_out;
#pragma unroll 1
  for (int col0 = t.rank * cols; col0 < filled; col0 += t.ranks * cols) {
    if (col0 != t.rank * cols) {
      __syncthreads();
      read_tile(col0);
      __syncthreads();
    }
#pragma unroll 2
    for (int i = t.tid; i < items; i += kThreads) {
      const int r = i >> p.cols_log2, col = col0 + (i & (cols - 1)), s = s_src[r];
      if (s < 0 || col >= (s_len[s] + kBS - 1) / kBS) continue;
      const bool swapped = s_uses[r] >= 0;
      if (in_place && s == r && !swapped) continue;
      p.tables_out[(int64_t)r * p.width + col] =
          swapped && col == s_len[s] / kBS ? s_part[r] : s_tile[i];
    }
  }
  if (alone && lead) {
    cg::this_cluster().barrier_wait();
    released.each_owned([&](int, int id) { q.extra_refs_out[id] = 0; });
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
  bool cluster;
  // workspace
  int32_t* same;    // [rows][list pieces] listed tokens that stay where they are, -1: the
                    // list is not one
  int32_t* counts;  // [pieces]
  uint32_t* masks;  // [pieces][kPer] entries that get a fresh block
  int32_t* fresh;   // [rows][width], of the changed blocks: the id that replaces it,
                    // INT_MIN: none does
};

__global__ void __launch_bounds__(kThreads, 1) compact_kernel(CompactK p) {
  extern __shared__ int sh[];
  const int R = p.num_rows;
  int* s_len = sh;            // old lengths
  int* s_start = sh + R;      // tokens kept as they are
  int* s_n = sh + 2 * R;      // tokens kept (-1: the row stays as it is)
  int* s_first = sh + 3 * R;  // first block that changes
  int* s_end = sh + 4 * R;    // 1: the list is not one; then the blocks popped up to and
                              // including the row
  __shared__ Scan scan;
  __shared__ int s_popped;
  const Team t(p.cluster);
  const bool lead = t.rank == 0;
  const Pool& q = p.pool;
  const int counted = *q.free_count;
  unsigned bad = 0;
  int longest = 0;
  const Largest of_lengths{scan.starts};
  for (int r = t.tid; r < R; r += kThreads) {
    const int64_t L = p.seq_lens[r];
    const int k = __ldg(p.keep_lens + r), start = p.keep_start ? __ldg(p.keep_start + r) : 0;
    const bool fits = L >= 0 && L <= (int64_t)p.width * kBS;
    const bool ok = fits && k <= p.max_keep && (k < 0 || (start >= 0 && start <= L - k));
    if (!ok) bad = PA_DEV_ERR_METADATA;
    s_len[r] = fits ? (int)L : 0;
    s_n[r] = ok && k >= 0 ? start + k : -1;
    s_start[r] = start;
    s_first[r] = s_end[r] = 0;
    longest = max(longest, s_len[r]);
  }
  of_lengths.put(t, longest);
  if (t.tid == 0) s_popped = 0;
  if (q.extra_refs != q.extra_refs_out) copy_refs(q, t);
  __syncthreads();
  const int filled = (of_lengths.get(t) + kBS - 1) / kBS;  // columns of the longest row
  // a piece of a row's table, and its blocks' further holders before the call
  const int segs = (max(filled, min(p.width, 1)) + kSeg - 1) / kSeg;  // (0: no columns)
  const int pieces = R * segs;
  auto look_up = [&](int i, int (&ids)[kPer], int (&extra)[kPer]) {
    const int r = i / segs, col0 = i % segs * kSeg, had = (s_len[r] + kBS - 1) / kBS;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int col = col0 + e * 32 + t.lane;
      ids[e] = s_n[r] >= 0 && col < had ? p.tables[(int64_t)r * p.width + col] : -1;
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      extra[e] = in_pool(q, ids[e]) ? __ldcg(q.extra_refs + ids[e]) : 0;
  };
  int first_ids[kPer], first_extra[kPer];  // (this warp's first, loaded ahead)
  if (t.gwarp < pieces) look_up(t.gwarp, first_ids, first_extra);
  // ---- the lists: ascending positions in [start, L); how many stay in place
  const int lsegs = (min(p.max_keep, p.width * kBS) + kSeg - 1) / kSeg;
  for (int i = t.gwarp; i < R * lsegs; i += t.gwarps) {
    const int r = i / lsegs, j0 = i % lsegs * kSeg;
    const int start = s_start[r], k = s_n[r] - start;
    if (s_n[r] < 0 || j0 >= k) continue;
    const int32_t* list = p.keep + (int64_t)r * p.max_keep;
    int v[kPer], before[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int j = j0 + e * 32 + t.lane;
      v[e] = j < k ? __ldg(list + j) : 0;
      before[e] = j < k && j > 0 ? __ldg(list + j - 1) : start - 1;
    }
    int same = 0;
    bool ok = true;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int j = j0 + e * 32 + t.lane;
      if (j >= k) break;
      ok = ok && v[e] > before[e] && v[e] < s_len[r];
      same += v[e] == start + j;
    }
    same = __reduce_add_sync(~0u, same);
    const bool all = __all_sync(~0u, ok);
    if (t.lane == 0) p.same[i] = all ? same : -1;
  }
  t.sync();
  for (int i = t.tid; i < R * lsegs; i += kThreads) {
    const int r = i / lsegs;
    if (s_n[r] < 0 || i % lsegs * kSeg >= s_n[r] - s_start[r]) continue;
    const int same = __ldcg(p.same + i);
    if (same < 0)
      s_end[r] = 1;
    else
      atomicAdd(&s_first[r], same);
  }
  __syncthreads();
  for (int r = t.tid; r < R; r += kThreads) {
    if (s_n[r] < 0) continue;
    if (s_end[r]) {
      bad = PA_DEV_ERR_METADATA;
      s_n[r] = -1;
    } else {
      s_first[r] = (s_start[r] + s_first[r]) / kBS;
    }
  }
  if (lead && bad) flag_error(q.err, bad);
  __syncthreads();
  // ---- blocks that change and have other holders: replaced by fresh ones
#pragma unroll 1
  for (int i = t.gwarp; i < pieces; i += t.gwarps) {
    const int r = i / segs, col0 = i % segs * kSeg;
    const int left = (s_n[r] + kBS - 1) / kBS, first = s_first[r];
    int n = 0;
    if (s_n[r] >= 0 && left > col0 && first < col0 + kSeg) {
      if (i != t.gwarp) look_up(i, first_ids, first_extra);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int col = col0 + e * 32 + t.lane;
        const bool changes = col >= first && col < left;
        if (changes && !in_pool(q, first_ids[e])) flag_error(q.err, PA_DEV_ERR_BLOCK_ID);
        const unsigned mask = __ballot_sync(~0u, changes && first_extra[e] > 0);
        n += __popc(mask);
        if (t.lane == 0) p.masks[i * kPer + e] = mask;
      }
    }
    if (t.lane == 0) p.counts[i] = n;
  }
  t.sync();
  // ---- pops in row order; the rows whose running need fits the stack run
  for (int64_t sum = 0, base = 0; base < pieces; base += kThreads) {
    const int i = (int)base + t.tid;
    const int n = i < pieces ? __ldcg(p.counts + i) : 0;
    const int64_t before = sum + block_scan_excl(n, &scan.total, scan.warp_sums);
    if (i < pieces && i % segs == segs - 1) s_end[i / segs] = (int)(before + n);
    sum += scan.total;
    __syncthreads();
  }
  const int64_t height = stack_height(q, counted, lead && t.tid == 0);
  bad = 0;
  for (int r = t.tid; r < R && pieces > 0; r += kThreads) {
    if (s_end[r] > height) {
      bad = PA_DEV_ERR_NO_BLOCKS;
      s_n[r] = -1;
    } else {
      atomicMax(&s_popped, s_end[r]);
    }
  }
  if (lead && bad) flag_error(q.err, bad);
  __syncthreads();
  const int64_t popped = s_popped;
  // ---- fresh ids
  for (int i = t.gwarp; i < pieces && popped > 0; i += t.gwarps) {  // (pieces without a pop)
    const int r = i / segs, col0 = i % segs * kSeg;
    if (s_n[r] < 0 || __ldcg(p.counts + i) != 0) continue;
    const int left = (s_n[r] + kBS - 1) / kBS;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int col = col0 + e * 32 + t.lane;
      if (col >= s_first[r] && col < left) p.fresh[(int64_t)r * p.width + col] = INT_MIN;
    }
  }
  if (popped > 0)
    in_order(t, pieces, p.counts, scan, [&](int i, int64_t before) {
      const int r = i / segs, col0 = i % segs * kSeg;
      if (s_n[r] < 0) return;
      const int left = (s_n[r] + kBS - 1) / kBS;
      const int32_t* row = p.tables + (int64_t)r * p.width;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int col = col0 + e * 32 + t.lane;
        const unsigned mask = __ldcg(p.masks + i * kPer + e);
        if (col >= s_first[r] && col < left) {
          int fresh = INT_MIN;
          if (mask >> t.lane & 1) {
            fresh = __ldcg(q.free_blocks +
                           (height - 1 - before - __popc(mask & ((1u << t.lane) - 1))));
            if (!in_pool(q, fresh)) {
              flag_error(q.err, PA_DEV_ERR_BLOCK_ID);
              fresh = -1;
            }
            atomicAdd(q.extra_refs_out + row[col], -1);
          }
          p.fresh[(int64_t)r * p.width + col] = fresh;
        }
        before += __popc(mask);
      }
    });
  // ---- a reference less for the blocks past the kept ones
  for (int i = t.gwarp; i < pieces; i += t.gwarps) {
    const int r = i / segs, col0 = i % segs * kSeg;
    const int had = (s_len[r] + kBS - 1) / kBS;
    const int left = max((s_n[r] + kBS - 1) / kBS, s_first[r]);
    if (s_n[r] < 0 || had <= col0 || left >= col0 + kSeg) continue;
    const int32_t* row = p.tables + (int64_t)r * p.width;
    int ids[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int col = col0 + e * 32 + t.lane;
      ids[e] = col >= left && col < had ? row[col] : -1;
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (in_pool(q, ids[e])) atomicAdd(q.extra_refs_out + ids[e], -1);
  }
  t.sync();
  auto load = [&](int r, int col0, int (&out)[kPer]) {
    const int had = (s_len[r] + kBS - 1) / kBS, n = s_n[r], left = (n + kBS - 1) / kBS;
    const int64_t at = (int64_t)r * p.width;
    // (nothing is replaced: only the blocks past the kept ones)
    const int from = n < 0 ? had : popped > 0 ? s_first[r] : max(s_first[r], left);
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int col = col0 + e * 32 + t.lane;
      out[e] = col >= from && col < had ? p.tables[at + col] : -1;
      if (col >= from && col < left && __ldcg(p.fresh + at + col) == INT_MIN) out[e] = -1;
    }
  };
  auto row_of = [](int r) { return r; };
  Released<decltype(load), decltype(row_of)> released(q, t, false, pieces, segs, p.width, load,
                                                      row_of);
  released.look_ahead();
  // ---- the moves: of a row that only loses its end none, unless its last block is
  // replaced.  (From the last warp on: the first ones have the released pieces.)
  const int64_t wide = (int64_t)p.max_keep + kBS;
  const int msegs = (int)((wide + kSeg - 1) / kSeg);
#pragma unroll 1
  for (int64_t i = t.gwarps - 1 - t.gwarp; i < (int64_t)R * msegs; i += t.gwarps) {
    const int r = (int)(i / msegs), j0 = (int)(i % msegs) * kSeg;
    const int n = s_n[r], at0 = s_first[r] * kBS, start = s_start[r];
    const int32_t* list = p.keep + (int64_t)r * p.max_keep;
    int moves = 0;
    if (n > at0) {
      // the last token stays where it is if and only if all do
      const bool whole = n == start || __ldg(list + (n - 1 - start)) == n - 1;
      const bool swapped =
          popped > 0 && __ldcg(p.fresh + (int64_t)r * p.width + s_first[r]) != INT_MIN;
      if (!whole || swapped) moves = n - at0;
    }
    if (j0 == 0 && t.lane == 0) {
      p.num_moves[r] = moves;
      p.seq_lens_out[r] = n >= 0 ? n : s_len[r];
    }
    const int32_t* row = p.tables + (int64_t)r * p.width;
    const int32_t* fresh = p.fresh + (int64_t)r * p.width;
    int pos[kPer], from[kPer], to[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int j = j0 + e * 32 + t.lane, at = at0 + j;
      pos[e] = j >= moves ? -1 : at < start ? at : __ldg(list + (at - start));
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int at = (at0 + j0 + e * 32 + t.lane) / kBS;
      from[e] = to[e] = 0;
      if (pos[e] >= 0) {
        from[e] = row[pos[e] / kBS];
        const int now = popped > 0 ? __ldcg(fresh + at) : INT_MIN;
        to[e] = now == INT_MIN ? row[at] : now;
      }
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      if (pos[e] < 0) continue;
      const int j = j0 + e * 32 + t.lane;
      const bool ok = in_pool(q, from[e]) && in_pool(q, to[e]);
      if (!ok) flag_error(q.err, PA_DEV_ERR_BLOCK_ID);
      p.src_slots[r * wide + j] = ok ? (int64_t)from[e] * kBS + pos[e] % kBS : -1;
      p.dst_slots[r * wide + j] = ok ? (int64_t)to[e] * kBS + (at0 + j) % kBS : -1;
    }
  }
  released.claim();
  // ---- the tables: out of place, whole
  const bool in_place = p.tables == p.tables_out;
  auto write_tables = [&]() {
#pragma unroll 1
    for (int i = t.gwarps - 1 - t.gwarp; i < pieces; i += t.gwarps) {
      const int r = i / segs, col0 = i % segs * kSeg;
      const int n = s_n[r], blocks = ((n >= 0 ? n : s_len[r]) + kBS - 1) / kBS;
      const int64_t at = (int64_t)r * p.width;
      int now[kPer], was[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int col = col0 + e * 32 + t.lane;
        const bool on = col < blocks;
        now[e] = on && popped > 0 && n >= 0 && col >= s_first[r] ? __ldcg(p.fresh + at + col)
                                                                 : INT_MIN;
        was[e] = on && !in_place ? p.tables[at + col] : 0;
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int col = col0 + e * 32 + t.lane;
        if (col < blocks && (now[e] != INT_MIN || !in_place))
          p.tables_out[at + col] = now[e] != INT_MIN ? now[e] : was[e];
      }
    }
  };
  if (!in_place) write_tables();
  t.sync();
  released.look_ahead();
  released.count(p.counts);
  t.sync();
  const int64_t freed = released.push(p.counts, height - popped, scan);
  if (lead && t.tid == 0)
    *q.free_count_out = (int)min(height - popped + freed, q.free_capacity);
  // ---- and in place what is replaced, once nobody reads the old ones
  if (in_place && popped > 0) {  // (the same in every CTA)
    t.sync();
    write_tables();
  }
}

// One kernel over `want` CTAs: a cluster of up to `team` where these are not too few, or a
// cooperative grid of at most one CTA per SM.  p.cluster tells the kernel which.
template <class P>
cudaError_t launch_team(void (*kernel)(P), P& p, int64_t want, size_t smem, size_t max_smem,
                        int num_sms, int team, cudaStream_t stream) {
  // (always the largest step's limit: see launch_build_step)
  static_assert(sizeof(Scan) < 20 * 1024, "with dynamic shared memory, 48 KB by default");
  if (smem > 28 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)max_smem);
    if (e != cudaSuccess) return e;
  }
  // (a cluster's barriers are shorter: 64 rows of 258 entries 14.5 us by 8 CTAs of one,
  // 18.4 by 9 of a grid; 64 rows of 513, compacted, 17.1 and 21.3 by 17.  16 CTAs where 9
  // to 24 are wanted: those two 13.1 -> 12.8 and 16.7 -> 15.4, 2 rows of 8192 entries 25
  // -> 16 us; where up to 48 or 80 are, a grid is faster, 31.8 against 36.4.)
  unsigned ctas = 1;
  const unsigned most = want > kMaxCluster ? team : kMaxCluster;
  while (ctas < most && ctas < want) ctas *= 2;
  p.cluster = want <= 3 * kMaxCluster;
  if (!p.cluster) ctas = (unsigned)(want < num_sms ? want : num_sms);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  if (p.cluster) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  } else {
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

Pool pool_of(const RowState& r, unsigned* err) {
  return Pool{r.extra_refs,    r.extra_refs_out, r.num_blocks,     r.free_blocks,
              r.free_capacity, r.free_count,     r.free_count_out, err};
}

int64_t pieces_of(int64_t rows, int64_t width) { return rows * ((width + kSeg - 1) / kSeg); }

// CTAs for a call: table entries, listed tokens and counts to copy, a few per thread
int64_t ctas_for(int64_t entries, int64_t listed, const RowState& r) {
  const int64_t copied = r.extra_refs == r.extra_refs_out ? 0 : r.num_blocks;
  const int64_t a = entries / (2 * kThreads), b = listed / (4 * kThreads),
                c = copied / (8 * kThreads);
  return 1 + (a > b ? (a > c ? a : c) : (b > c ? b : c));
}

constexpr size_t kTileBytes = 64 * 1024;  // of a tile of the new tables, at most

}  // namespace

int largest_team() {
  int fewest = 1;
  auto query = [&](auto kernel) {
    const int smem = (int)(5 * kMaxForkRows * 4 + kTileBytes);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kBigCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kBigCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
            cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();  // (not this device, then)
      n = 0;
    }
    fewest = n < fewest ? n : fewest;
  };
  query(fork_kernel);
  query(compact_kernel);
  return fewest > 0 ? kBigCluster : kMaxCluster;
}

int64_t fork_workspace_bytes(int num_rows, int max_blocks_per_seq) {
  return 4 * (num_rows + pieces_of(num_rows, max_blocks_per_seq));
}

cudaError_t launch_fork_blocks(const ForkArgs& a, int num_sms, int team, cudaStream_t stream) {
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
  p.row_need = static_cast<int32_t*>(a.workspace);
  p.counts = p.row_need + R;
  const int64_t want = ctas_for(R * p.width, 0, a.rows);
  // columns of a tile: a line of 32, fewer (a sector of 8) where that spreads the
  // columns over more CTAs, and what fits at the largest numbers of rows
  p.cols_log2 = 5;
  while (p.cols_log2 > 3 && (int64_t)p.width <= want << (p.cols_log2 - 1)) --p.cols_log2;
  while (p.cols_log2 > 0 && ((size_t)R * 4) << p.cols_log2 > kTileBytes) --p.cols_log2;
  return launch_team(fork_kernel, p, want, (size_t)(5 + (1 << p.cols_log2)) * R * 4,
                     (size_t)5 * kMaxForkRows * 4 + kTileBytes, num_sms, team, stream);
}

int64_t compact_workspace_bytes(int num_rows, int max_blocks_per_seq) {
  return 4 * (pieces_of(num_rows, (int64_t)max_blocks_per_seq * kBS) +
              (1 + kPer) * pieces_of(num_rows, max_blocks_per_seq) +
              (int64_t)num_rows * max_blocks_per_seq);
}

cudaError_t launch_compact_blocks(const CompactArgs& a, int num_sms, int team,
                                  cudaStream_t stream) {
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
  p.same = static_cast<int32_t*>(a.workspace);
  p.counts = p.same + pieces_of(R, (int64_t)p.width * kBS);
  p.masks = reinterpret_cast<uint32_t*>(p.counts + pieces_of(R, p.width));
  p.fresh = reinterpret_cast<int32_t*>(p.masks) + kPer * pieces_of(R, p.width);
  return launch_team(compact_kernel, p, ctas_for(R * p.width, R * (int64_t)p.max_keep, a.rows),
                     (size_t)(5 * R * 4), (size_t)5 * kMaxForkRows * 4 + kTileBytes, num_sms, team,
                     stream);
}

}  // namespace pa
