// The decode attention of causal rows (kv4_decode.cuh).
#include "kv4_decode.cuh"

namespace grg {

size_t kv4_decode_counter_bytes() { return kCounterBytes; }
size_t kv4_decode_partial_bytes(int rows, int head_dim) {
  return static_cast<size_t>(kPartialSlots) * rows * (head_dim * 4 + 8);
}

template int launch_kv4_decode<false>(const Kv4AttnArgs& a, int max_packed_rows, size_t counters_at,
                                      bool f16, cudaStream_t stream);

}  // namespace grg
