// Arguments and launchers of the operators around a layer's LoRA products
// (internal): norm, append to the 4-bit cache, attention over it.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace grg {

struct NormArgs {
  const uint16_t* x;
  long long x_stride;
  const uint16_t* residual;  // null: none
  long long residual_stride;
  const uint16_t* weight;
  float eps;
  int hidden;
  uint16_t* residual_out;  // null: not wanted
  long long residual_out_stride;
  uint16_t* y;  // null: not wanted
  long long y_stride;
  uint8_t* y8;  // null: not wanted
  long long y8_stride;
  float* y8_scale;
  int group;  // columns per scale: hidden or 128
  const int32_t* num_tokens;
  int max_num_tokens;
  uint32_t* status;  // null: not wanted
};
int launch_add_rmsnorm(const NormArgs& a, bool f16, cudaStream_t stream);

struct Kv4AppendArgs {
  const uint16_t* q;  // null: no q
  long long q_stride;
  uint16_t* q_out;
  long long q_out_stride;
  const uint16_t* k;
  long long k_stride;
  const uint16_t* v;
  long long v_stride;
  const float* rope;  // null: no rotation
  int max_positions;
  int rope_dim;
  int interleaved;
  const int32_t* positions;
  const int32_t* slots;
  uint8_t* cache;
  long long num_slots;  // num_pages * page_size
  int num_q_heads;      // 0 without q
  int num_kv_heads;
  int page_size;
  int head_dim;
  float k_scale;
  float v_scale;
  float inv_k_scale;
  float inv_v_scale;
  uint16_t* k_held;  // null: not wanted
  uint16_t* v_held;
  const int32_t* num_tokens;
  int max_num_tokens;
  uint32_t* status;
};
int launch_kv4_append(const Kv4AppendArgs& a, bool f16, cudaStream_t stream);

struct Kv4AttnArgs {
  const uint16_t* q;
  long long q_stride;
  uint16_t* out;
  long long out_stride;
  float* lse;  // null: not wanted
  const uint8_t* cache;
  int num_pages;
  int num_q_heads;
  int num_kv_heads;
  int page_size;
  int head_dim;
  float score_scale;  // softmax_scale * k_scale
  float v_scale;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* page_table;
  long long table_stride;
  int num_seqs;
  int max_num_tokens;
  int max_q_len;
  int window;  // 0: none
  const uint32_t* tree_mask;  // [max_num_tokens][tree_words], null for causal rows
  int tree_words;
  int short_rows;  // trees of up to so many packed rows over up to so many keys go by the decode kernel
  int short_keys;
  void* workspace;
  uint32_t* status;
};
size_t kv4_attention_workspace(long long num_seqs, long long max_num_tokens, long long max_q_len,
                               int num_q_heads, int num_kv_heads, int head_dim);
int launch_kv4_attention(const Kv4AttnArgs& a, bool f16, cudaStream_t stream);

struct Kv4AcceptArgs {
  uint8_t* cache;
  int num_pages;
  int num_kv_heads;
  int page_size;
  int head_dim;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* page_table;
  long long table_stride;
  int num_seqs;
  const int32_t* path;  // [num_seqs][max_path]
  const int32_t* path_len;
  int max_path;
  int32_t* kv_len_out;
  uint32_t* status;
};
int launch_kv4_accept(const Kv4AcceptArgs& a, cudaStream_t stream);

struct Kv4WeightsArgs {
  float* weights;  // [num_seqs][num_kv_heads][capacity]
  int capacity;
  const uint16_t* q;
  long long q_stride;
  const float* lse;  // [max_num_tokens][num_q_heads]
  const uint8_t* cache;
  int num_pages;
  int num_q_heads;
  int num_kv_heads;
  int page_size;
  int head_dim;
  float score_scale;  // softmax_scale * k_scale
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* page_table;
  long long table_stride;
  int num_seqs;
  int max_num_tokens;
  int max_q_len;
  int window;           // 0: none
  const int32_t* path;  // [num_seqs][max_path], null: a sequence's rows are all of its own
  const int32_t* path_len;
  int max_path;
  uint32_t* status;
};
int launch_kv4_weights(const Kv4WeightsArgs& a, bool f16, cudaStream_t stream);

struct Kv4EvictArgs {
  uint8_t* cache;
  int num_pages;
  int num_kv_heads;
  int page_size;
  int head_dim;
  float* weights;    // [num_seqs][num_kv_heads][capacity]
  int32_t* key_pos;  // the same
  int capacity;
  const int32_t* kv_len;
  const int32_t* last_pos;
  const int32_t* page_table;
  long long table_stride;
  int num_seqs;
  int budget;
  int sink;
  int recent;
  int32_t* kv_len_out;
  uint32_t* status;
  int smem_keys;  // the launcher's: keys whose integers are kept in shared memory, and pages
  int smem_pages;
  int cluster;  // CTAs of a head
  unsigned long long page_magic;  // ceil(2^36 / blocks of a page)
};
int launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t stream);

}  // namespace grg
