// step_kernels.cu -- a step's metadata on the GPU (pa_build_step).
//
// From each request's query length n and computed length c:
//   need_r = ceil((c + n) / 16) - ceil(c / 16) new blocks, popped from a stack
//   of free ids in request order; request r runs if the needs and the query
//   lengths up to and including its own fit the stack and the token arrays
//   (both sums only grow, so the requests that run are a prefix);
//   query_start_loc = running sum of n, position = c + i, slot =
//   table[position / 16] * 16 + position % 16 ("vLLM engine anatomy", Figure 2).
//
// A few hundred KB at most move, so the call is bound by launch latency and
// the dependent loads, not by bandwidth: one launch of one cluster.  Every CTA
// scans all requests for itself (their lengths are a few KB that L2 holds),
// keeps the sums in shared memory and fills its share of the tokens and of the
// new table entries, so no second kernel waits for the sums.  64 decodes 4.3 us,
// 1000 decodes and four chunks of 2047 tokens 6.4 us.
#include <cooperative_groups.h>

#include "pa_step.cuh"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kStepThreads = 1024;
// tokens plus requests one CTA fills before the cluster grows: two passes of
// its threads
constexpr int kStepPerCta = 2 * kStepThreads;
constexpr int kStepMaxCluster = 8;  // the portable cluster size

struct StepArgs {
  const int32_t* query_lens;
  const int32_t* computed_lens;
  int num_seqs;
  int32_t* block_tables;
  int max_blocks_per_seq;
  const int32_t* free_blocks;
  int64_t free_capacity;
  const int32_t* free_count;
  int32_t* free_count_out;
  int64_t num_blocks, num_tokens;
  int32_t* seq_lens;
  int32_t* query_start_loc;
  int32_t* positions;
  int64_t* slot_mapping;
  unsigned* err;
};

// largest r in [0, n) with a[r] <= x (a non-decreasing, a[0] <= x)
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kStepThreads) build_step_kernel(StepArgs p) {
  extern __shared__ int sh[];
  int* s_start = sh;                   // first query token of request r
  int* s_before = sh + p.num_seqs;     // new blocks of the requests before r
  int* s_done = sh + 2 * p.num_seqs;   // computed length
  __shared__ long long warp_sums[32];
  __shared__ long long total[2];       // one iteration's sums: tokens, blocks
  __shared__ int s_tokens, s_blocks;   // of the requests that run
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), nranks = (int)cl.num_blocks();
  const int tid = threadIdx.x;
  const bool lead = rank == 0;
  int64_t free_n = *p.free_count;  // (free_count_out may be the same word)
  unsigned bad = 0;
  if (free_n < 0 || free_n > p.free_capacity) {
    bad = PA_DEV_ERR_METADATA;
    free_n = 0;
  }
  if (tid == 0) s_tokens = s_blocks = 0;
  const int64_t table_keys = (int64_t)p.max_blocks_per_seq * kBS;
  long long sum_n = 0, sum_need = 0;
  for (int base = 0; base < p.num_seqs; base += kStepThreads) {
    const int r = base + tid;
    long long n = 0, c = 0, need = 0;
    if (r < p.num_seqs) {
      n = p.query_lens[r];
      c = p.computed_lens[r];
      if (c < 0 || c > table_keys) {
        bad |= PA_DEV_ERR_METADATA;
        n = c = 0;
      } else if (n < 0 || c + n > table_keys) {
        bad |= PA_DEV_ERR_METADATA;
        n = 0;
      }
      need = (c + n + kBS - 1) / kBS - (c + kBS - 1) / kBS;
    }
    const long long n0 = sum_n + block_scan_excl(n, &total[0], warp_sums);
    const long long b0 = sum_need + block_scan_excl(need, &total[1], warp_sums);
    sum_n += total[0];
    sum_need += total[1];
    if (r < p.num_seqs) {
      const bool room = b0 + need <= free_n;
      const bool fits = n0 + n <= p.num_tokens;
      if (!room) bad |= PA_DEV_ERR_NO_BLOCKS;
      if (!fits) bad |= PA_DEV_ERR_METADATA;
      const bool runs = room && fits;
      if (runs) {
        atomicMax(&s_tokens, (int)(n0 + n));
        atomicMax(&s_blocks, (int)(b0 + need));
      }
      // requests that do not run start behind the last one that does
      s_start[r] = runs ? (int)n0 : 0x7fffffff;
      s_before[r] = runs ? (int)b0 : 0x7fffffff;
      s_done[r] = (int)c;
    }
    __syncthreads();  // total[] is written again by the next iteration
  }
  if (lead && bad) flag_error(p.err, bad);
  // every length and the stack's height are read: outputs may replace them
  cl.sync();
  const int tokens = s_tokens, blocks = s_blocks;
  const int64_t gtid = (int64_t)rank * kStepThreads + tid;
  const int64_t gsize = (int64_t)nranks * kStepThreads;
  if (lead && tid == 0) {
    *p.free_count_out = (int)(free_n - blocks);
    p.query_start_loc[p.num_seqs] = tokens;
  }
  for (int64_t r = gtid; r < p.num_seqs; r += gsize) {
    const int start = min(s_start[r], tokens);
    const int next = r + 1 < p.num_seqs ? min(s_start[r + 1], tokens) : tokens;
    p.query_start_loc[r] = start;
    p.seq_lens[r] = s_done[r] + (next - start);
  }
  for (int64_t i = gtid; i < blocks; i += gsize) {
    const int r = last_at_most(s_before, p.num_seqs, (int)i);
    const int col = (s_done[r] + kBS - 1) / kBS + (int)i - s_before[r];
    const int id = __ldg(p.free_blocks + (free_n - 1 - i));
    p.block_tables[(int64_t)r * p.max_blocks_per_seq + col] = id;
  }
  for (int64_t t = gtid; t < p.num_tokens; t += gsize) {
    int pos = 0;
    int64_t slot = -1;
    if (t < tokens) {
      const int r = last_at_most(s_start, p.num_seqs, (int)t);
      pos = s_done[r] + (int)t - s_start[r];
      const int have = (s_done[r] + kBS - 1) / kBS, b = pos / kBS;
      // a block the request held already, or the one popped for it
      const int id =
          b < have ? p.block_tables[(int64_t)r * p.max_blocks_per_seq + b]
                   : __ldg(p.free_blocks + (free_n - 1 - (s_before[r] + b - have)));
      if (id >= 0 && (int64_t)id < p.num_blocks)
        slot = (int64_t)id * kBS + pos % kBS;
      else
        flag_error(p.err, PA_DEV_ERR_BLOCK_ID);
    }
    p.positions[t] = pos;
    p.slot_mapping[t] = slot;
  }
}

}  // namespace

cudaError_t launch_build_step(const int32_t* query_lens, const int32_t* computed_lens,
                              int num_seqs, int32_t* block_tables,
                              int max_blocks_per_seq, const int32_t* free_blocks,
                              int64_t free_capacity, const int32_t* free_count,
                              int32_t* free_count_out, int64_t num_blocks,
                              int64_t num_tokens, int32_t* seq_lens,
                              int32_t* query_start_loc, int32_t* positions,
                              int64_t* slot_mapping, unsigned* err,
                              cudaStream_t stream) {
  StepArgs p{query_lens,  computed_lens, num_seqs,   block_tables, max_blocks_per_seq,
             free_blocks, free_capacity, free_count, free_count_out, num_blocks,
             num_tokens,  seq_lens,      query_start_loc, positions, slot_mapping,
             err};
  const int64_t work = num_tokens + num_seqs;
  int cluster = 1;
  while (cluster < kStepMaxCluster && (int64_t)cluster * kStepPerCta < work) cluster *= 2;
  const size_t smem = (size_t)3 * num_seqs * sizeof(int);
  // Steps that may not fit the default 48 KB, of which the kernel's static shared
  // memory takes some 300 bytes.  Always the same limit, the largest step's: one of
  // each call's own size could be lowered by another thread before this launch.
  if (smem > 40 * 1024) {
    constexpr int kMaxSmem = 3 * kMaxBuildSeqs * (int)sizeof(int);
    const cudaError_t e = cudaFuncSetAttribute(
        build_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)cluster);
  cfg.blockDim = dim3(kStepThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, build_step_kernel, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace pa
