// The decode attention of rows of drafted trees (kv4_decode.cuh).
#include "kv4_decode.cuh"

namespace grg {

template int launch_kv4_decode<true>(const Kv4AttnArgs& a, int max_packed_rows, size_t counters_at,
                                     bool f16, cudaStream_t stream);

}  // namespace grg
