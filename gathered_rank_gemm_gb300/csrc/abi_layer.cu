// The C ABI of the operators around a layer's LoRA products: argument checks
// and dispatch.  Declarations and the full contract live in
// include/gathered_rank_gemm.h.
#include <cmath>
#include <cstdint>

#include "gathered_rank_gemm.h"
#include "layer.h"

namespace {

bool aligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
bool stride_ok(int64_t stride, int64_t width) { return stride >= width && stride < (1ll << 40); }
bool factor_ok(float s) { return std::isfinite(s) && s > 0.0f && std::isfinite(1.0f / s); }
bool tokens_ok(int64_t n) { return n >= 1 && n <= LORA_MAX_NUM_TOKENS; }

int add_rmsnorm(const uint16_t* x, int64_t x_row_stride, const uint16_t* residual,
                int64_t residual_row_stride, const uint16_t* weight, float eps, int64_t hidden,
                uint16_t* residual_out, int64_t residual_out_row_stride, uint16_t* y,
                int64_t y_row_stride, uint8_t* y8, int64_t y8_row_stride, float* y8_scale,
                int64_t group, const int32_t* num_tokens, int64_t max_num_tokens,
                uint32_t* status, void* stream, bool f16) {
  if (!x || !weight || !num_tokens || (!y && !y8 && !residual_out) || (y8 && !y8_scale))
    return LORA_ERR_NULL;
  if (hidden < 8 || hidden > LORA_NORM_MAX_HIDDEN || hidden % 8 != 0 ||
      !tokens_ok(max_num_tokens) || !(eps >= 0.0f) || !std::isfinite(eps))
    return LORA_ERR_SHAPE;
  if (y8 && group != hidden && (group != 128 || hidden % 128 != 0)) return LORA_ERR_SHAPE;
  if (!stride_ok(x_row_stride, hidden) || (residual && !stride_ok(residual_row_stride, hidden)) ||
      (residual_out && !stride_ok(residual_out_row_stride, hidden)) ||
      (y && !stride_ok(y_row_stride, hidden)) || (y8 && !stride_ok(y8_row_stride, hidden)))
    return LORA_ERR_SHAPE;
  if (!aligned(x, 16) || x_row_stride % 8 || !aligned(weight, 16) || !aligned(num_tokens, 4) ||
      (residual && (!aligned(residual, 16) || residual_row_stride % 8)) ||
      (residual_out && (!aligned(residual_out, 16) || residual_out_row_stride % 8)) ||
      (y && (!aligned(y, 16) || y_row_stride % 8)) ||
      (y8 && (!aligned(y8, 8) || y8_row_stride % 8 || !aligned(y8_scale, 4))) ||
      !aligned(status, 4))
    return LORA_ERR_ALIGN;
  grg::NormArgs a;
  a.x = x;
  a.x_stride = x_row_stride;
  a.residual = residual;
  a.residual_stride = residual_row_stride;
  a.weight = weight;
  a.eps = eps;
  a.hidden = static_cast<int>(hidden);
  a.residual_out = residual_out;
  a.residual_out_stride = residual_out_row_stride;
  a.y = y;
  a.y_stride = y_row_stride;
  a.y8 = y8;
  a.y8_stride = y8_row_stride;
  a.y8_scale = y8_scale;
  a.group = static_cast<int>(y8 ? group : hidden);
  a.num_tokens = num_tokens;
  a.max_num_tokens = static_cast<int>(max_num_tokens);
  a.status = status;
  return grg::launch_add_rmsnorm(a, f16, static_cast<cudaStream_t>(stream));
}

// Sizes that the append and the attention share.
bool cache_ok(int64_t num_pages, int num_kv_heads, int page_size, int head_dim) {
  return (head_dim == 64 || head_dim == 128) && num_kv_heads >= 1 &&
         num_kv_heads <= LORA_KV4_MAX_HEADS && page_size >= 16 &&
         page_size <= LORA_KV4_MAX_PAGE_SIZE && page_size % 16 == 0 && num_pages >= 1 &&
         num_pages < (1ll << 31) / page_size;
}

int kv4_append(const uint16_t* q, int64_t q_row_stride, uint16_t* q_out, int64_t q_out_row_stride,
               int num_q_heads, const uint16_t* k, int64_t k_row_stride, const uint16_t* v,
               int64_t v_row_stride, const float* rope, int64_t max_positions, int rope_dim,
               int interleaved, const int32_t* positions, const int32_t* slots, uint8_t* cache,
               int64_t num_pages, int num_kv_heads, int page_size, int head_dim, float k_scale,
               float v_scale, uint16_t* k_held, uint16_t* v_held, const int32_t* num_tokens,
               int64_t max_num_tokens, uint32_t* status, void* stream, bool f16) {
  if (!k || !v || !slots || !cache || !num_tokens || (q && !q_out) || (rope && !positions))
    return LORA_ERR_NULL;
  if (!cache_ok(num_pages, num_kv_heads, page_size, head_dim) || !tokens_ok(max_num_tokens) ||
      !factor_ok(k_scale) || !factor_ok(v_scale))
    return LORA_ERR_SHAPE;
  if (q && (num_q_heads < 1 || num_q_heads > LORA_KV4_MAX_HEADS)) return LORA_ERR_SHAPE;
  if (rope && (max_positions < 1 || max_positions > (1ll << 31) - 1 || rope_dim < 32 ||
               rope_dim > head_dim || rope_dim % 32 != 0))
    return LORA_ERR_SHAPE;
  const int64_t qw = static_cast<int64_t>(num_q_heads) * head_dim;
  const int64_t kw = static_cast<int64_t>(num_kv_heads) * head_dim;
  if ((q && (!stride_ok(q_row_stride, qw) || !stride_ok(q_out_row_stride, qw))) ||
      !stride_ok(k_row_stride, kw) || !stride_ok(v_row_stride, kw))
    return LORA_ERR_SHAPE;
  if ((q && (!aligned(q, 16) || q_row_stride % 8 || !aligned(q_out, 16) || q_out_row_stride % 8)) ||
      !aligned(k, 16) || k_row_stride % 8 || !aligned(v, 16) || v_row_stride % 8 ||
      !aligned(rope, 16) || !aligned(positions, 4) || !aligned(slots, 4) || !aligned(cache, 16) ||
      !aligned(k_held, 16) || !aligned(v_held, 16) || !aligned(num_tokens, 4) ||
      !aligned(status, 4))
    return LORA_ERR_ALIGN;
  grg::Kv4AppendArgs a;
  a.q = q;
  a.q_stride = q_row_stride;
  a.q_out = q_out;
  a.q_out_stride = q_out_row_stride;
  a.k = k;
  a.k_stride = k_row_stride;
  a.v = v;
  a.v_stride = v_row_stride;
  a.rope = rope;
  a.max_positions = static_cast<int>(max_positions);
  a.rope_dim = rope_dim;
  a.interleaved = interleaved;
  a.positions = positions;
  a.slots = slots;
  a.cache = cache;
  a.num_slots = num_pages * page_size;
  a.num_q_heads = q ? num_q_heads : 0;
  a.num_kv_heads = num_kv_heads;
  a.page_size = page_size;
  a.head_dim = head_dim;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.inv_k_scale = 1.0f / k_scale;
  a.inv_v_scale = 1.0f / v_scale;
  a.k_held = k_held;
  a.v_held = v_held;
  a.num_tokens = num_tokens;
  a.max_num_tokens = static_cast<int>(max_num_tokens);
  a.status = status;
  return grg::launch_kv4_append(a, f16, static_cast<cudaStream_t>(stream));
}

bool path_ok(int64_t max_path) { return max_path >= 1 && max_path <= LORA_KV4_MAX_PATH; }
bool capacity_ok(int64_t capacity) { return capacity >= 1 && capacity <= LORA_KV4_MAX_KEYS; }
bool seqs_ok(int64_t num_seqs) { return num_seqs >= 1 && num_seqs <= LORA_KV4_MAX_SEQS; }
// Whether an array of n words and one of m have one in common.
bool overlap(const void* a, int64_t n, const void* b, int64_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(m) * 4 && y < x + static_cast<uintptr_t>(n) * 4;
}
bool table_ok(int64_t table_stride, int page_size) {
  return table_stride >= 1 && table_stride < (1ll << 31) / page_size;
}

bool attention_sizes_ok(int64_t num_seqs, int64_t max_num_tokens, int64_t max_q_len,
                        int num_q_heads, int num_kv_heads, int head_dim) {
  return num_seqs >= 1 && num_seqs <= LORA_KV4_MAX_SEQS && tokens_ok(max_num_tokens) &&
         max_q_len >= 1 && max_q_len <= max_num_tokens && (head_dim == 64 || head_dim == 128) &&
         num_kv_heads >= 1 && num_kv_heads <= LORA_KV4_MAX_HEADS && num_q_heads >= 1 &&
         num_q_heads <= LORA_KV4_MAX_HEADS && num_q_heads % num_kv_heads == 0;
}

int kv4_attention(const uint16_t* q, int64_t q_row_stride, uint16_t* out, int64_t out_row_stride,
                  float* lse, int num_q_heads, const uint8_t* cache, int64_t num_pages,
                  int num_kv_heads, int page_size, int head_dim, float k_scale, float v_scale,
                  const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table,
                  int64_t table_stride, int64_t num_seqs, int64_t max_num_tokens,
                  int64_t max_q_len, float softmax_scale, int64_t window, const uint32_t* tree_mask,
                  int tree_words, void* workspace, size_t workspace_bytes, uint32_t* status,
                  void* stream, bool f16) {
  if (!q || !out || !cache || !q_start || !kv_len || !page_table || !workspace)
    return LORA_ERR_NULL;
  if (!cache_ok(num_pages, num_kv_heads, page_size, head_dim) ||
      !attention_sizes_ok(num_seqs, max_num_tokens, max_q_len, num_q_heads, num_kv_heads,
                          head_dim) ||
      !factor_ok(k_scale) || !factor_ok(v_scale) || !std::isfinite(softmax_scale) ||
      !(softmax_scale > 0.0f) || !(softmax_scale * k_scale > 0.0f) ||
      !std::isfinite(softmax_scale * k_scale) || window < 0 || window >= (1ll << 31) ||
      !table_ok(table_stride, page_size))
    return LORA_ERR_SHAPE;
  const int64_t qw = static_cast<int64_t>(num_q_heads) * head_dim;
  if (!stride_ok(q_row_stride, qw) || !stride_ok(out_row_stride, qw)) return LORA_ERR_SHAPE;
  if (!aligned(q, 16) || q_row_stride % 8 || !aligned(out, 16) || out_row_stride % 8 ||
      !aligned(lse, 4) || !aligned(cache, 16) || !aligned(q_start, 4) || !aligned(kv_len, 4) ||
      !aligned(page_table, 4) || !aligned(tree_mask, 4) || !aligned(workspace, 16) ||
      !aligned(status, 4))
    return LORA_ERR_ALIGN;
  if (workspace_bytes < grg::kv4_attention_workspace(num_seqs, max_num_tokens, max_q_len,
                                                     num_q_heads, num_kv_heads, head_dim))
    return LORA_ERR_WORKSPACE;
  grg::Kv4AttnArgs a;
  a.q = q;
  a.q_stride = q_row_stride;
  a.out = out;
  a.out_stride = out_row_stride;
  a.lse = lse;
  a.cache = cache;
  a.num_pages = static_cast<int>(num_pages);
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.page_size = page_size;
  a.head_dim = head_dim;
  a.score_scale = softmax_scale * k_scale;
  a.v_scale = v_scale;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.table_stride = table_stride;
  a.num_seqs = static_cast<int>(num_seqs);
  a.max_num_tokens = static_cast<int>(max_num_tokens);
  a.max_q_len = static_cast<int>(max_q_len);
  a.window = static_cast<int>(window);
  a.tree_mask = tree_mask;
  a.tree_words = tree_words;
  a.short_rows = a.short_keys = 0;
  a.workspace = workspace;
  a.status = status;
  return grg::launch_kv4_attention(a, f16, static_cast<cudaStream_t>(stream));
}

int kv4_key_weights(float* weights, int64_t capacity, const uint16_t* q, int64_t q_row_stride,
                    const float* lse, int num_q_heads, const uint8_t* cache, int64_t num_pages,
                    int num_kv_heads, int page_size, int head_dim, float k_scale,
                    const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table,
                    int64_t table_stride, int64_t num_seqs, int64_t max_num_tokens,
                    int64_t max_q_len, float softmax_scale, int64_t window, const int32_t* path,
                    const int32_t* path_len, int64_t max_path, uint32_t* status, void* stream,
                    bool f16) {
  if (!weights || !q || !lse || !cache || !q_start || !kv_len || !page_table ||
      (path != nullptr) != (path_len != nullptr))
    return LORA_ERR_NULL;
  if (!cache_ok(num_pages, num_kv_heads, page_size, head_dim) ||
      !attention_sizes_ok(num_seqs, max_num_tokens, max_q_len, num_q_heads, num_kv_heads,
                          head_dim) ||
      !factor_ok(k_scale) || !std::isfinite(softmax_scale) || !(softmax_scale > 0.0f) ||
      !(softmax_scale * k_scale > 0.0f) || !std::isfinite(softmax_scale * k_scale) || window < 0 ||
      window >= (1ll << 31) || !table_ok(table_stride, page_size) || !capacity_ok(capacity) ||
      (path && !path_ok(max_path)))
    return LORA_ERR_SHAPE;
  if (!stride_ok(q_row_stride, static_cast<int64_t>(num_q_heads) * head_dim)) return LORA_ERR_SHAPE;
  if (!aligned(weights, 4) || !aligned(q, 16) || q_row_stride % 8 || !aligned(lse, 4) ||
      !aligned(cache, 16) || !aligned(q_start, 4) || !aligned(kv_len, 4) ||
      !aligned(page_table, 4) || !aligned(path, 4) || !aligned(path_len, 4) || !aligned(status, 4))
    return LORA_ERR_ALIGN;
  grg::Kv4WeightsArgs a;
  a.weights = weights;
  a.capacity = static_cast<int>(capacity);
  a.q = q;
  a.q_stride = q_row_stride;
  a.lse = lse;
  a.cache = cache;
  a.num_pages = static_cast<int>(num_pages);
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.page_size = page_size;
  a.head_dim = head_dim;
  a.score_scale = softmax_scale * k_scale;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.table_stride = table_stride;
  a.num_seqs = static_cast<int>(num_seqs);
  a.max_num_tokens = static_cast<int>(max_num_tokens);
  a.max_q_len = static_cast<int>(max_q_len);
  a.window = static_cast<int>(window);
  a.path = path;
  a.path_len = path_len;
  a.max_path = path ? static_cast<int>(max_path) : 0;
  a.status = status;
  return grg::launch_kv4_weights(a, f16, static_cast<cudaStream_t>(stream));
}

}  // namespace

#pragma GCC visibility push(default)
extern "C" {

#define GRG_NORM(name, half)                                                                      \
  int name(const uint16_t* x, int64_t x_row_stride, const uint16_t* residual,                     \
           int64_t residual_row_stride, const uint16_t* weight, float eps, int64_t hidden,        \
           uint16_t* residual_out, int64_t residual_out_row_stride, uint16_t* y,                  \
           int64_t y_row_stride, uint8_t* y8, int64_t y8_row_stride, float* y8_scale,             \
           int64_t group, const int32_t* num_tokens, int64_t max_num_tokens, uint32_t* status,    \
           void* stream) {                                                                        \
    return add_rmsnorm(x, x_row_stride, residual, residual_row_stride, weight, eps, hidden,       \
                       residual_out, residual_out_row_stride, y, y_row_stride, y8, y8_row_stride, \
                       y8_scale, group, num_tokens, max_num_tokens, status, stream, half);        \
  }
GRG_NORM(lora_add_rmsnorm, false)
GRG_NORM(lora_add_rmsnorm_f16, true)
#undef GRG_NORM

#define GRG_APPEND(name, half)                                                                    \
  int name(const uint16_t* q, int64_t q_row_stride, uint16_t* q_out, int64_t q_out_row_stride,    \
           int num_q_heads, const uint16_t* k, int64_t k_row_stride, const uint16_t* v,           \
           int64_t v_row_stride, const float* rope, int64_t max_positions, int rope_dim,          \
           int interleaved, const int32_t* positions, const int32_t* slots, uint8_t* cache,       \
           int64_t num_pages, int num_kv_heads, int page_size, int head_dim, float k_scale,       \
           float v_scale, uint16_t* k_held, uint16_t* v_held, const int32_t* num_tokens,          \
           int64_t max_num_tokens, uint32_t* status, void* stream) {                              \
    return kv4_append(q, q_row_stride, q_out, q_out_row_stride, num_q_heads, k, k_row_stride, v,  \
                      v_row_stride, rope, max_positions, rope_dim, interleaved, positions, slots, \
                      cache, num_pages, num_kv_heads, page_size, head_dim, k_scale, v_scale,      \
                      k_held, v_held, num_tokens, max_num_tokens, status, stream, half);          \
  }
GRG_APPEND(lora_kv4_append, false)
GRG_APPEND(lora_kv4_append_f16, true)
#undef GRG_APPEND

size_t lora_kv4_attention_workspace_size(int64_t num_seqs, int64_t max_num_tokens,
                                         int64_t max_q_len, int num_q_heads, int num_kv_heads,
                                         int head_dim) {
  if (!attention_sizes_ok(num_seqs, max_num_tokens, max_q_len, num_q_heads, num_kv_heads,
                          head_dim))
    return 0;
  return grg::kv4_attention_workspace(num_seqs, max_num_tokens, max_q_len, num_q_heads,
                                      num_kv_heads, head_dim);
}

#define GRG_ATTENTION(name, half)                                                                 \
  int name(const uint16_t* q, int64_t q_row_stride, uint16_t* out, int64_t out_row_stride,        \
           float* lse, int num_q_heads, const uint8_t* cache, int64_t num_pages,                  \
           int num_kv_heads, int page_size, int head_dim, float k_scale, float v_scale,           \
           const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table,              \
           int64_t table_stride, int64_t num_seqs, int64_t max_num_tokens, int64_t max_q_len,     \
           float softmax_scale, int64_t window, void* workspace, size_t workspace_bytes,          \
           uint32_t* status, void* stream) {                                                      \
    return kv4_attention(q, q_row_stride, out, out_row_stride, lse, num_q_heads, cache,           \
                         num_pages, num_kv_heads, page_size, head_dim, k_scale, v_scale, q_start, \
                         kv_len, page_table, table_stride, num_seqs, max_num_tokens, max_q_len,   \
                         softmax_scale, window, nullptr, 0, workspace, workspace_bytes, status,   \
                         stream, half);                                                           \
  }
GRG_ATTENTION(lora_kv4_attention, false)
GRG_ATTENTION(lora_kv4_attention_f16, true)
#undef GRG_ATTENTION

#define GRG_TREE(name, half)                                                                      \
  int name(const uint16_t* q, int64_t q_row_stride, uint16_t* out, int64_t out_row_stride,        \
           float* lse, int num_q_heads, const uint8_t* cache, int64_t num_pages,                  \
           int num_kv_heads, int page_size, int head_dim, float k_scale, float v_scale,           \
           const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table,              \
           int64_t table_stride, int64_t num_seqs, int64_t max_num_tokens, int64_t max_q_len,     \
           const uint32_t* tree_mask, int64_t mask_words, float softmax_scale, int64_t window,    \
           void* workspace, size_t workspace_bytes, uint32_t* status, void* stream) {             \
    if (!tree_mask) return LORA_ERR_NULL;                                                         \
    if (mask_words < 1 || mask_words > LORA_MAX_NUM_TOKENS / 32 || 32 * mask_words < max_q_len)   \
      return LORA_ERR_SHAPE;                                                                      \
    return kv4_attention(q, q_row_stride, out, out_row_stride, lse, num_q_heads, cache,           \
                         num_pages, num_kv_heads, page_size, head_dim, k_scale, v_scale, q_start, \
                         kv_len, page_table, table_stride, num_seqs, max_num_tokens, max_q_len,   \
                         softmax_scale, window, tree_mask, static_cast<int>(mask_words),          \
                         workspace, workspace_bytes, status, stream, half);                       \
  }
GRG_TREE(lora_kv4_tree_attention, false)
GRG_TREE(lora_kv4_tree_attention_f16, true)
#undef GRG_TREE

#define GRG_WEIGHTS(name, half)                                                                   \
  int name(float* weights, int64_t capacity, const uint16_t* q, int64_t q_row_stride,             \
           const float* lse, int num_q_heads, const uint8_t* cache, int64_t num_pages,            \
           int num_kv_heads, int page_size, int head_dim, float k_scale, const int32_t* q_start,  \
           const int32_t* kv_len, const int32_t* page_table, int64_t table_stride,                \
           int64_t num_seqs, int64_t max_num_tokens, int64_t max_q_len, float softmax_scale,      \
           int64_t window, const int32_t* path, const int32_t* path_len, int64_t max_path,        \
           uint32_t* status, void* stream) {                                                      \
    return kv4_key_weights(weights, capacity, q, q_row_stride, lse, num_q_heads, cache,           \
                           num_pages, num_kv_heads, page_size, head_dim, k_scale, q_start,        \
                           kv_len, page_table, table_stride, num_seqs, max_num_tokens, max_q_len, \
                           softmax_scale, window, path, path_len, max_path, status, stream,       \
                           half);                                                                 \
  }
GRG_WEIGHTS(lora_kv4_key_weights, false)
GRG_WEIGHTS(lora_kv4_key_weights_f16, true)
#undef GRG_WEIGHTS

int lora_kv4_accept(uint8_t* cache, int64_t num_pages, int num_kv_heads, int page_size, int head_dim,
                    const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table,
                    int64_t table_stride, int64_t num_seqs, const int32_t* path,
                    const int32_t* path_len, int64_t max_path, int32_t* kv_len_out,
                    uint32_t* status, void* stream) {
  if (!cache || !q_start || !kv_len || !page_table || !path || !path_len || !kv_len_out)
    return LORA_ERR_NULL;
  if (!cache_ok(num_pages, num_kv_heads, page_size, head_dim) || !seqs_ok(num_seqs) ||
      !table_ok(table_stride, page_size) || !path_ok(max_path) ||
      overlap(kv_len, num_seqs, kv_len_out, num_seqs) ||
      overlap(path_len, num_seqs, kv_len_out, num_seqs) ||
      overlap(q_start, num_seqs + 1, kv_len_out, num_seqs) ||
      overlap(path, num_seqs * max_path, kv_len_out, num_seqs) ||
      overlap(page_table, num_seqs * table_stride, kv_len_out, num_seqs))
    return LORA_ERR_SHAPE;
  if (!aligned(cache, 16) || !aligned(q_start, 4) || !aligned(kv_len, 4) ||
      !aligned(page_table, 4) || !aligned(path, 4) || !aligned(path_len, 4) ||
      !aligned(kv_len_out, 4) || !aligned(status, 4))
    return LORA_ERR_ALIGN;
  grg::Kv4AcceptArgs a;
  a.cache = cache;
  a.num_pages = static_cast<int>(num_pages);
  a.num_kv_heads = num_kv_heads;
  a.page_size = page_size;
  a.head_dim = head_dim;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.table_stride = table_stride;
  a.num_seqs = static_cast<int>(num_seqs);
  a.path = path;
  a.path_len = path_len;
  a.max_path = static_cast<int>(max_path);
  a.kv_len_out = kv_len_out;
  a.status = status;
  return grg::launch_kv4_accept(a, static_cast<cudaStream_t>(stream));
}

int lora_kv4_evict(uint8_t* cache, int64_t num_pages, int num_kv_heads, int page_size, int head_dim,
                   float* weights, int32_t* key_pos, int64_t capacity, const int32_t* kv_len,
                   const int32_t* last_pos, const int32_t* page_table, int64_t table_stride,
                   int64_t num_seqs, int64_t budget, int64_t sink, int64_t recent,
                   int32_t* kv_len_out, uint32_t* status, void* stream) {
  if (!cache || !weights || !key_pos || !kv_len || !last_pos || !page_table || !kv_len_out)
    return LORA_ERR_NULL;
  if (!cache_ok(num_pages, num_kv_heads, page_size, head_dim) || !seqs_ok(num_seqs) ||
      !table_ok(table_stride, page_size) || !capacity_ok(capacity) || budget < 1 ||
      budget >= (1ll << 31) || sink < 0 || recent < 0 || sink > budget || recent > budget - sink ||
      overlap(kv_len, num_seqs, kv_len_out, num_seqs) ||
      overlap(last_pos, num_seqs, kv_len_out, num_seqs) ||
      overlap(page_table, num_seqs * table_stride, kv_len_out, num_seqs) ||
      overlap(weights, num_seqs * num_kv_heads * capacity, kv_len_out, num_seqs) ||
      overlap(key_pos, num_seqs * num_kv_heads * capacity, kv_len_out, num_seqs))
    return LORA_ERR_SHAPE;
  if (!aligned(cache, 16) || !aligned(weights, 4) || !aligned(key_pos, 4) || !aligned(kv_len, 4) ||
      !aligned(last_pos, 4) || !aligned(page_table, 4) || !aligned(kv_len_out, 4) ||
      !aligned(status, 4))
    return LORA_ERR_ALIGN;
  grg::Kv4EvictArgs a;
  a.cache = cache;
  a.num_pages = static_cast<int>(num_pages);
  a.num_kv_heads = num_kv_heads;
  a.page_size = page_size;
  a.head_dim = head_dim;
  a.weights = weights;
  a.key_pos = key_pos;
  a.capacity = static_cast<int>(capacity);
  a.kv_len = kv_len;
  a.last_pos = last_pos;
  a.page_table = page_table;
  a.table_stride = table_stride;
  a.num_seqs = static_cast<int>(num_seqs);
  a.budget = static_cast<int>(budget);
  a.sink = static_cast<int>(sink);
  a.recent = static_cast<int>(recent);
  a.kv_len_out = kv_len_out;
  a.status = status;
  a.smem_keys = a.smem_pages = a.cluster = 0;
  return grg::launch_kv4_evict(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
#pragma GCC visibility pop
