// pa_beam.h -- host-side interfaces between the C ABI (pa_api.cu) and the
// kernels of decoding with several hypotheses: beam selection, forked and
// compacted rows, copies and moves over the caches of all layers.
#pragma once

#include "pa_internal.h"

namespace pa {

// ---- beam selection (beam_kernels.cu) ---------------------------------------
constexpr int kMaxBeams = 64;          // beams of one group
constexpr int kMaxVocab = 1 << 24;
constexpr int kMaxBeamSelected = 128;  // continuations of one group
constexpr int kBeamThreads = 256;
constexpr int kBeamAlign = 8;  // a row may start up to 7 elements into 16 bytes
struct BeamPlan {
  int per_thread;             // logits of one thread of a chunk
  int chunks;                 // of a row
  int64_t off_stats, bytes;   // workspace: keys, then each chunk's (max, sum)
};
BeamPlan make_beam_plan(pa_dtype dtype, int num_groups, int beam_width, int vocab_size,
                        int num_selected);
int64_t beam_workspace_bytes(int num_groups, int beam_width, int vocab_size, int num_selected);
struct BeamArgs {
  const void* logits;
  pa_dtype dtype;
  int num_groups, beam_width, vocab_size;
  int64_t row_stride;
  const float* beam_scores;
  const uint8_t* finished;
  int end_token;
  int num_selected;
  float* scores;
  int32_t* parents;
  int32_t* tokens;
  uint8_t* finished_out;
  void* workspace;
};
cudaError_t launch_beam_select(const BeamArgs& a, const BeamPlan& plan, int num_sms,
                               cudaStream_t stream);

// ---- forked and compacted rows (fork_kernels.cu) ------------------------------
// rows of one call: five ints each in one CTA's shared memory
constexpr int kMaxForkRows = 4096;
// table entries of one call: their places and INT_MIN make the claims of freed blocks
constexpr int64_t kMaxForkEntries = 1ll << 30;
// what both calls read and change; an _out may be its input
struct RowState {
  int num_rows;
  const int32_t* block_tables;
  int32_t* block_tables_out;
  int max_blocks_per_seq;
  const int32_t* seq_lens;
  int32_t* seq_lens_out;
  const int32_t* extra_refs;
  int32_t* extra_refs_out;
  int64_t num_blocks;
  int32_t* free_blocks;
  int64_t free_capacity;
  const int32_t* free_count;
  int32_t* free_count_out;
};
struct ForkArgs {
  RowState rows;
  const int32_t* sources;
  int64_t* block_mapping;
  int32_t* num_pairs;
  void* workspace;
  unsigned* err;
};
int64_t fork_workspace_bytes(int num_rows, int max_blocks_per_seq);
// CTAs of the largest cluster that the current device holds of both calls' kernels
int largest_team();
cudaError_t launch_fork_blocks(const ForkArgs& a, int num_sms, int team, cudaStream_t stream);

struct CompactArgs {
  RowState rows;
  const int32_t* keep;
  int max_keep;
  const int32_t* keep_lens;
  const int32_t* keep_start;  // null: 0
  int64_t* src_slots;         // [rows][max_keep + 16]
  int64_t* dst_slots;
  int32_t* num_moves;
  void* workspace;
  unsigned* err;
};
int64_t compact_workspace_bytes(int num_rows, int max_blocks_per_seq);
cudaError_t launch_compact_blocks(const CompactArgs& a, int num_sms, int team,
                                  cudaStream_t stream);

// ---- copies and moves of all layers (move_kernels.cu) --------------------------
struct LayerCaches {
  void* k;
  void* v;
  int64_t k_layer_bytes, v_layer_bytes;  // from one layer to the next
  int num_layers;
  int64_t num_blocks;
  int num_kv_heads;
  pa_dtype dtype;
  int head_dim;
};
cudaError_t launch_copy_blocks_layers(const LayerCaches& c, int64_t block_bytes,
                                      const int64_t* block_mapping, int64_t max_pairs,
                                      const int32_t* num_pairs, int num_sms, unsigned* err,
                                      cudaStream_t stream);
cudaError_t launch_move_tokens(const LayerCaches& c, const int64_t* src_slots,
                               const int64_t* dst_slots, const int32_t* num_moves,
                               int num_rows, int64_t max_moves, int num_sms, unsigned* err,
                               cudaStream_t stream);

}  // namespace pa
