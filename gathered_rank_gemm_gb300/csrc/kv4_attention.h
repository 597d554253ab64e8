// The kernels behind lora_kv4_attention (internal).
#pragma once

#include "layer.h"

namespace grg {

// Sequences with at most max_packed_rows rows x heads of a key head (kv4_decode.cu).
int launch_kv4_decode(const Kv4AttnArgs& a, int max_packed_rows, bool f16, cudaStream_t stream);
// Its workspace for groups of `rows` (8 or 16) packed rows.
size_t kv4_decode_workspace(int rows, int head_dim);

// Sequences with more than that (kv4_prefill.cu).
int launch_kv4_prefill(const Kv4AttnArgs& a, int max_packed_rows, bool f16, cudaStream_t stream);

}  // namespace grg
