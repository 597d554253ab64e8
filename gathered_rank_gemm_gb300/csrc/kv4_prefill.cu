// The prefill attention of causal rows (kv4_prefill.cuh), and which kernel takes what.
#include <algorithm>

#include "kv4_prefill.cuh"

namespace grg {

namespace {
// Sequences of up to kDecodeRows packed rows take the decode kernel, the others
// the prefill kernel; a batch whose bound allows no long sequence does not launch
// the latter.  Measured, by the decode and by the prefill kernel: 48 windows of 2048
// keys with up to 30 packed rows of 64 20.2 and 55.4 us; 64 sequences of 2000 keys with 32
// packed rows of 128 110 and 131 us, with 64 186 and 131 us; 16 of 2000 with 48 rows 55.1
// and 48.0 us.
constexpr int kDecodeRows = 32;
// Trees of few sequences go by the decode kernel up to kTreeRows packed rows, where every group of
// 16 rows and every key head has an SM of its own and the keys of all groups together are at most
// kTreeWork (kTreeWork64 for heads of 64): one tree of 15 rows, 32 / 8
// heads of 128, over 700 keys 11.6 us, 21.6 us by the prefill kernel; over 32000 55.6 and 66.0; over
// 64000 88.9 and 85.2; four trees (128 groups) over 6000 keys 38.8 and 42.4, over 8000 48.7 and 46.9;
// heads of 64, 128 groups over 700 keys 11.2 and 16.7, over 4000 30.6 and 24.2.
constexpr int kTreeRows = 256;  // (the decode kernel's division of packed rows)
constexpr long long kTreeWork = 800000, kTreeWork64 = 300000;

long long packed_bound(long long max_q_len, int num_q_heads, int num_kv_heads) {
  return max_q_len * (num_q_heads / num_kv_heads);
}
size_t prefill_partials(int head_dim) {
  return static_cast<size_t>(2) * kPreCtasMax * kPreRows * (head_dim * 4 + 8);
}
}  // namespace

// The workspace: the two kernels' counters, then partials, which the kernels of a
// call use one after the other.
size_t kv4_attention_workspace(long long, long long, long long max_q_len, int num_q_heads,
                               int num_kv_heads, int head_dim) {
  const long long packed = packed_bound(max_q_len, num_q_heads, num_kv_heads);
  size_t n = kv4_decode_partial_bytes(packed > 8 ? 16 : 8, head_dim);
  if (packed > kDecodeRows) n = max(n, prefill_partials(head_dim));
  return kPreCounterBytes + kv4_decode_counter_bytes() + n;
}

template int launch_kv4_prefill<false>(const Kv4AttnArgs& a, int max_packed_rows, bool f16,
                                       cudaStream_t stream);
extern template int launch_kv4_prefill<true>(const Kv4AttnArgs& a, int max_packed_rows, bool f16,
                                             cudaStream_t stream);  // kv4_prefill_tree.cu

namespace {
template <bool TREE>
int launch_both(const Kv4AttnArgs& a, bool f16, cudaStream_t stream) {
  const int rc = launch_kv4_decode<TREE>(a, kDecodeRows, kPreCounterBytes, f16, stream);
  if (rc != 0) return rc;
  return packed_bound(a.max_q_len, a.num_q_heads, a.num_kv_heads) > kDecodeRows
             ? launch_kv4_prefill<TREE>(a, kDecodeRows, f16, stream)
             : 0;
}
}  // namespace

int launch_kv4_attention(const Kv4AttnArgs& a, bool f16, cudaStream_t stream) {
  if (!a.tree_mask) return launch_both<false>(a, f16, stream);
  Kv4AttnArgs b = a;
  const long long packed = packed_bound(a.max_q_len, a.num_q_heads, a.num_kv_heads);
  const long long items = (std::min<long long>(packed, kTreeRows) + 15) / 16 * a.num_seqs * a.num_kv_heads;
  b.short_rows = items <= device_sm_count() ? kTreeRows : 0;
  b.short_keys = static_cast<int>((a.head_dim == 64 ? kTreeWork64 : kTreeWork) / items);
  if (packed <= b.short_rows && a.table_stride * a.page_size <= b.short_keys)
    return launch_kv4_decode<true>(b, kDecodeRows, kPreCounterBytes, f16, stream);
  return launch_both<true>(b, f16, stream);
}

}  // namespace grg
