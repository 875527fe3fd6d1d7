// pa_step.h -- host-side interfaces between the C ABI (pa_api.cu) and the
// kernels of a sparse decode step: metadata, norm + rotation + cache write,
// block bounds and selection, attention over selected blocks.
#pragma once

#include "pa_internal.h"

namespace pa {

// ---- a step's metadata (step_kernels.cu) ------------------------------------
// requests of one pa_build_step: three ints each in one CTA's shared memory
constexpr int kMaxBuildSeqs = 16384;
cudaError_t launch_build_step(const int32_t* query_lens, const int32_t* computed_lens,
                              int num_seqs, int32_t* block_tables,
                              int max_blocks_per_seq, const int32_t* free_blocks,
                              int64_t free_capacity, const int32_t* free_count,
                              int32_t* free_count_out, int64_t num_blocks,
                              int64_t num_tokens, int32_t* seq_lens,
                              int32_t* query_start_loc, int32_t* positions,
                              int64_t* slot_mapping, unsigned* err,
                              cudaStream_t stream);

// ---- norm, rotation and cache write (rope_kernels.cuh) ----------------------
struct RopeArgs {
  const void* q;
  const void* k;
  const void* v;
  pa_dtype dtype;
  int64_t num_tokens, q_stride, k_stride, v_stride;
  const void* q_weight;  // null: no norm
  const void* k_weight;
  pa_dtype weight_dtype;  // dtype or PA_F32
  float eps;
  const float* cos_sin;  // [max_position][rotary_dim]
  int64_t max_position;
  int rotary_dim, interleaved;
  const int32_t* positions;
  void* q_out;
  void* k_cache;
  void* v_cache;
  pa_dtype cache_dtype;
  int64_t num_blocks;
  int num_q_heads, num_kv_heads, head_dim;
  const int64_t* slot_mapping;
  float k_scale, v_scale;
  bool vector_ok;  // q, k, v rows and the weights allow 16-byte loads
};
cudaError_t launch_norm_rope_and_cache(const RopeArgs& a, int num_sms, unsigned* err,
                                       cudaStream_t stream);

// ---- block bounds and selection (select_kernels.cu) -------------------------
struct StepView {  // a step's metadata, as pa_attention takes it
  const int32_t* block_tables;
  int max_blocks_per_seq;
  const int32_t* seq_lens;
  const int32_t* query_start_loc;
  int num_seqs;
  int64_t num_tokens;
  int max_query_len, max_seq_len;
  int64_t num_blocks;
  unsigned* err;
};
cudaError_t launch_summarise_blocks(const StepView& s, const void* k_cache,
                                    pa_dtype cache_dtype, int num_kv_heads,
                                    int head_dim, void* bounds, cudaStream_t stream);

// scores of the tokens of one pass over the step: room for as many tokens as
// kSelectScoreBytes hold, one token at least
constexpr int64_t kSelectScoreBytes = 48ll << 20;
constexpr int64_t kSelectPassTokens = 32768;  // of a pass at most (grid.y)
struct SelectPlan {
  int64_t row_scores;   // scores of one (token, KV head): blocks, a multiple of 4
  int64_t pass_tokens;  // tokens of one pass
  int64_t bytes;
};
SelectPlan make_select_plan(int64_t num_tokens, int num_kv_heads, int max_seq_len);
cudaError_t launch_select_blocks(const StepView& s, const SelectPlan& plan,
                                 const void* q, pa_dtype q_dtype, int num_q_heads,
                                 int num_kv_heads, int head_dim, const void* bounds,
                                 int max_selected, int keep_first, int keep_last,
                                 int32_t* selected, int32_t* num_selected,
                                 void* workspace, int num_sms, cudaStream_t stream);

// ---- attention over selected blocks (attn_selected.cu) ----------------------
struct SelectedPlan {
  int head_rows;   // query heads of one KV head that a CTA takes
  int head_parts;  // CTAs per share, where the group has more
  int64_t shares;  // equal shares of all the lists' entries
  int64_t off_ml, off_cut, bytes;  // workspace
};
SelectedPlan make_selected_plan(pa_dtype cache_dtype, int64_t num_tokens, int num_q_heads,
                                int num_kv_heads, int head_dim, int max_selected,
                                int num_sms);
struct SelectedArgs {
  const void* q;
  pa_dtype q_dtype;
  const void* k_cache;
  const void* v_cache;
  pa_dtype cache_dtype;
  int num_q_heads, num_kv_heads, head_dim;
  const int32_t* selected;
  const int32_t* num_selected;
  int max_selected;
  float scale, k_scale, v_scale;
  void* out;
  void* workspace;
};
cudaError_t launch_attention_selected(const StepView& s, const SelectedPlan& plan,
                                      const SelectedArgs& a, cudaStream_t stream);

}  // namespace pa
