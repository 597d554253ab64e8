// The accepted path of a drafted tree moves together in the 4-bit cache:
//   new[n - m + i] = old[n - m + path[i]],  i < path_len,
// for the n keys of a sequence whose last m are the tree's.
//
// Every entry of a head is read before any is written, so a path may name rows in any order,
// and one row twice.  A CTA has a few heads of a sequence: a short path's entries (up to
// kAcceptShort) wait in registers, a head a warp; a long one's in shared memory, a head at a
// time.  Bound by a chain of latencies: lengths, path, page, entry.
#include <algorithm>

#include "kv4_move.cuh"
#include "launch.h"
#include "layer.h"

namespace grg {

namespace {
constexpr int kAcceptWarps = 8;
constexpr int kAcceptShort = 16;
}

template <int D>
__global__ void __launch_bounds__(kAcceptWarps * 32, 4)
    lora_kv4_accept_kernel(const __grid_constant__ Kv4AcceptArgs a) {
  using Entry = Kv4Entry<D>;
  constexpr int LANES = Entry::kLanes, SHORT = kAcceptShort * LANES / 32;  // units of a lane
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int b = blockIdx.x, head0 = blockIdx.y * warps;
  pdl_wait();
  pdl_launch_dependents();

  const int q0 = a.q_start[b], q1 = a.q_start[b + 1], n0 = a.kv_len[b], len0 = a.path_len[b];
  const int room = static_cast<int>(a.table_stride) * a.page_size;  // below 2^31
  const int n = min(max(n0, 0), room);
  const long long drafted = static_cast<long long>(q1) - q0;
  const int m = static_cast<int>(min(max(drafted, 0ll), static_cast<long long>(n)));
  const int len = min(max(len0, 0), min(m, a.max_path));
  bool odd = n != n0 || m != drafted || len != len0, lost = false;
  const int base = n - m;
  if (head0 == 0 && tid == 0) a.kv_len_out[b] = base + len;
  const int32_t* path = a.path + static_cast<long long>(b) * a.max_path;
  const Kv4Pages pages{a.cache, a.page_table + b * a.table_stride, a.num_pages, a.num_kv_heads, a.page_size};
  // Where entry i of the path comes from and goes to (null: it stays, or a page is not there),
  // and its place in the block.
  struct Move {
    uint8_t *source, *target;
    int from, to;
  };
  auto move_of = [&](int i, int h) {
    Move x{nullptr, nullptr, 0, base + i};
    const int c = i < len ? __ldg(path + i) : i;
    if (c == i) return x;
    if (c < 0 || c >= m) {
      odd = true;
      return x;
    }
    x.from = base + c;
    x.source = pages.block<D>(x.from, h);
    x.target = pages.block<D>(x.to, h);
    if (!x.source || !x.target) {
      lost = true;
      x.source = nullptr;
    }
    return x;
  };

  if (len <= kAcceptShort) {
    const int h = head0 + warp;
    if (h < a.num_kv_heads && len > 0) {
      Move x[SHORT];
      Entry e[SHORT];
      const int part = lane % LANES;
#pragma unroll
      for (int u = 0; u < SHORT; ++u) x[u] = move_of((u * 32 + lane) / LANES, h);
#pragma unroll
      for (int u = 0; u < SHORT; ++u)
        if (x[u].source) e[u].load(x[u].source, x[u].from % 16, part);  // (page_size is a multiple of 16)
      __syncwarp();
#pragma unroll
      for (int u = 0; u < SHORT; ++u)
        if (x[u].source) e[u].store(x[u].target, x[u].to % 16, part);
    }
  } else {
    Entry* staged = reinterpret_cast<Entry*>(smem);
    for (int h = head0; h < min(head0 + warps, a.num_kv_heads); ++h) {
      for (int u = tid; u < len * LANES; u += blockDim.x) {
        const Move x = move_of(u / LANES, h);
        if (x.source) staged[u].load(x.source, x.from % 16, u % LANES);
      }
      __syncthreads();
      for (int u = tid; u < len * LANES; u += blockDim.x) {
        const Move x = move_of(u / LANES, h);
        if (x.source) staged[u].store(x.target, x.to % 16, u % LANES);
      }
      __syncthreads();
    }
  }
  if (a.status) {
    if (odd) atomicOr(a.status, kStatusBadLength);
    if (lost) atomicOr(a.status, kStatusBadSlot);
  }
}

int launch_kv4_accept(const Kv4AcceptArgs& a, cudaStream_t stream) {
  const bool wide = a.head_dim == 128;
  const void* fn = wide ? reinterpret_cast<const void*>(lora_kv4_accept_kernel<128>)
                        : reinterpret_cast<const void*>(lora_kv4_accept_kernel<64>);
  const size_t smem = a.max_path <= kAcceptShort ? 0
                      : static_cast<size_t>(a.max_path) * (wide ? Kv4Entry<128>::kLanes * sizeof(Kv4Entry<128>)
                                                                : Kv4Entry<64>::kLanes * sizeof(Kv4Entry<64>));
  if (ensure_smem_attr(fn, smem) != 0) return -6;
  const int warps = std::min(kAcceptWarps, a.num_kv_heads);
  Kv4AcceptArgs p = a;
  return launch_pdl(fn, dim3(a.num_seqs, (a.num_kv_heads + warps - 1) / warps), dim3(warps * 32), smem,
                    stream, 0, &p);
}

}  // namespace grg
