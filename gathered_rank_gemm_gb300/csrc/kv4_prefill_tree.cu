// The prefill attention of rows of drafted trees (kv4_prefill.cuh).
#include "kv4_prefill.cuh"

namespace grg {

template int launch_kv4_prefill<true>(const Kv4AttnArgs& a, int max_packed_rows, bool f16,
                                      cudaStream_t stream);

}  // namespace grg
