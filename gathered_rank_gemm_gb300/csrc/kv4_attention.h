// The kernels behind lora_kv4_attention (internal).
#pragma once

#include "layer.h"

namespace grg {

// Sequences with at most max_packed_rows rows x heads of a key head
// (kv4_decode.cuh).  Its counters lie at counters_at in the workspace, its
// partials behind them.  TREE: rows see what their masks name.
template <bool TREE>
int launch_kv4_decode(const Kv4AttnArgs& a, int max_packed_rows, size_t counters_at, bool f16,
                      cudaStream_t stream);
size_t kv4_decode_counter_bytes();
size_t kv4_decode_partial_bytes(int rows, int head_dim);  // groups of 8 or 16 packed rows

// Sequences with more than that (kv4_prefill.cuh).
template <bool TREE>
int launch_kv4_prefill(const Kv4AttnArgs& a, int max_packed_rows, bool f16, cudaStream_t stream);

}  // namespace grg
