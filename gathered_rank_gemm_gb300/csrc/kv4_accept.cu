// The accepted path of a drafted tree moves together in the 4-bit cache:
//   new[n - m + i] = old[n - m + path[i]],  i < path_len,
// for the n keys of a sequence whose last m are the tree's.
//
// Every entry of a head is read before any is written, so a path may name rows in any order,
// and one row twice.  A warp has a head of a sequence; the entries wait in shared memory.
// Bound by a chain of latencies: lengths, path, page, entry.
#include "kv4_move.cuh"
#include "launch.h"
#include "layer.h"

namespace grg {

namespace {
constexpr int kAcceptWarps = 8;
}

template <int D>
__global__ void __launch_bounds__(kAcceptWarps * 32)
    lora_kv4_accept_kernel(const __grid_constant__ Kv4AcceptArgs a) {
  using Entry = Kv4Entry<D>;
  constexpr int LANES = Entry::kLanes;
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = blockDim.x >> 5;
  const int h = blockIdx.y * warps + warp, b = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  if (h >= a.num_kv_heads) return;

  const int q0 = a.q_start[b], q1 = a.q_start[b + 1], n0 = a.kv_len[b], len0 = a.path_len[b];
  const int room = static_cast<int>(a.table_stride) * a.page_size;  // below 2^31
  const int n = min(max(n0, 0), room);
  const int m = static_cast<int>(min(max(static_cast<long long>(q1) - q0, 0ll), static_cast<long long>(n)));
  const int len = min(max(len0, 0), min(m, a.max_path));
  bool odd = n != n0 || m != static_cast<long long>(q1) - q0 || len != len0, lost = false;
  const int base = n - m;
  const int32_t* path = a.path + static_cast<long long>(b) * a.max_path;
  const Kv4Pages pages{a.cache, a.page_table + b * a.table_stride, a.num_pages, a.num_kv_heads, a.page_size};
  Entry* staged = reinterpret_cast<Entry*>(smem) + static_cast<size_t>(warp) * a.max_path * LANES;

  const int units = len * LANES;  // (entry, lane of it)
  for (int u = lane; u < units; u += 32) {
    const int i = u / LANES, part = u % LANES, c = __ldg(path + i);
    if (c == i) continue;
    if (c < 0 || c >= m) {
      odd = true;
      continue;
    }
    const uint8_t* from = pages.block<D>(base + c, h);
    if (from) staged[u].load(from, (base + c) % 16, part);  // (page_size is a multiple of 16)
    else lost = true;
  }
  __syncwarp();
  for (int u = lane; u < units; u += 32) {
    const int i = u / LANES, part = u % LANES, c = __ldg(path + i);
    if (c == i || c < 0 || c >= m || !pages.block<D>(base + c, h)) continue;
    uint8_t* to = pages.block<D>(base + i, h);
    if (to) staged[u].store(to, (base + i) % 16, part);
    else lost = true;
  }
  if (h == 0 && lane == 0) a.kv_len_out[b] = base + len;
  if (a.status) {
    if (odd) atomicOr(a.status, kStatusBadLength);
    if (lost) atomicOr(a.status, kStatusBadSlot);
  }
}

int launch_kv4_accept(const Kv4AcceptArgs& a, cudaStream_t stream) {
  const bool wide = a.head_dim == 128;
  const void* fn = wide ? reinterpret_cast<const void*>(lora_kv4_accept_kernel<128>)
                        : reinterpret_cast<const void*>(lora_kv4_accept_kernel<64>);
  const size_t each = static_cast<size_t>(a.max_path) *
                      (wide ? Kv4Entry<128>::kLanes * sizeof(Kv4Entry<128>)
                            : Kv4Entry<64>::kLanes * sizeof(Kv4Entry<64>));
  int warps = kAcceptWarps;
  while (warps > 1 && (warps * each > 96 * 1024 || warps / 2 >= a.num_kv_heads)) warps /= 2;
  const size_t smem = warps * each;
  if (ensure_smem_attr(fn, smem) != 0) return -6;
  Kv4AcceptArgs p = a;
  return launch_pdl(fn, dim3(a.num_seqs, (a.num_kv_heads + warps - 1) / warps), dim3(warps * 32), smem,
                    stream, 0, &p);
}

}  // namespace grg
