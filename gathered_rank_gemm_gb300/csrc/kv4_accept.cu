// The accepted path of a drafted tree moves together in the 4-bit cache:
//   new[n - m + i] = old[n - m + path[i]],  i < path_len,
// for the n keys of a sequence whose last m are the tree's.
//
// Every entry of a head is read before any is written, so a path may name rows in any order,
// and one row twice.  A warp has a head of a sequence and moves eight entries at a time through
// registers.  In a path that ascends no entry comes from where an earlier one went, so that its
// eights follow one another; of others, only those of up to eight go this way, and the rest wait
// in shared memory, a head at a time.  Bound by a chain of latencies: lengths, path, page, entry
// (15 rows of one sequence, 8 heads 2.4 us; 256 sequences, 32 heads 6.6 us, four heads a warp 8.9 us).
#include <algorithm>

#include "kv4_move.cuh"
#include "launch.h"
#include "layer.h"

namespace grg {

namespace {
constexpr int kAcceptWarps = 8;
constexpr int kAcceptOnce = 8;   // entries that a warp moves at a time
}

template <int D>
__global__ void __launch_bounds__(kAcceptWarps * 32, 3)
    lora_kv4_accept_kernel(const __grid_constant__ Kv4AcceptArgs a) {
  using Entry = Kv4Entry<D>;
  constexpr int LANES = Entry::kLanes, UNITS = kAcceptOnce * LANES / 32;  // entries' pieces of a lane: 2 or 1
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
  const long long head_bytes = static_cast<long long>(a.page_size / 16) * Kv4Block<D>::kBytes;
  // Where entry i of the path comes from and goes to in the first head (null: it stays, or a page is
  // not there), and its place in the block.
  struct Move {
    uint8_t *source, *target;
    int from, to;
  };
  auto move_of = [&](int i) {
    Move x{nullptr, nullptr, 0, base + i};
    const int c = i < len ? __ldg(path + i) : i;
    if (c == i) return x;
    if (c < 0 || c >= m) {
      odd = true;
      return x;
    }
    x.from = base + c;
    x.source = pages.block<D>(x.from, 0);
    x.target = pages.block<D>(x.to, 0);
    if (!x.source || !x.target) {
      lost = true;
      x.source = nullptr;
    }
    return x;
  };
  bool falls = false;  // (rows that are none move nothing)
  if (len > kAcceptOnce)
    for (int i = lane; i < len - 1; i += 32) {
      const int c = __ldg(path + i), d = __ldg(path + i + 1);
      falls = falls || !(c < d && c >= 0 && d < m);
    }
  falls = __any_sync(0xffffffffu, falls);  // (the same in every warp)

  if (!falls) {
    const int h = head0 + warp, part = lane % LANES;
    for (int i0 = 0; h < a.num_kv_heads && i0 < len; i0 += kAcceptOnce) {
      Move x[UNITS];
      Entry e[UNITS];
#pragma unroll
      for (int u = 0; u < UNITS; ++u) x[u] = move_of(i0 + (u * 32 + lane) / LANES);
#pragma unroll
      for (int u = 0; u < UNITS; ++u)  // (page_size is a multiple of 16)
        if (x[u].source) e[u].load(x[u].source + h * head_bytes, x[u].from % 16, part);
      __syncwarp();
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
        if (x[u].source) e[u].store(x[u].target + h * head_bytes, x[u].to % 16, part);
      __syncwarp();
    }
  } else {
    Entry* staged = reinterpret_cast<Entry*>(smem);
    for (int h = head0; h < min(head0 + warps, a.num_kv_heads); ++h) {
      for (int u = tid; u < len * LANES; u += blockDim.x) {
        const Move x = move_of(u / LANES);
        if (x.source) staged[u].load(x.source + h * head_bytes, x.from % 16, u % LANES);
      }
      __syncthreads();
      for (int u = tid; u < len * LANES; u += blockDim.x) {
        const Move x = move_of(u / LANES);
        if (x.source) staged[u].store(x.target + h * head_bytes, x.to % 16, u % LANES);
      }
      __syncthreads();
    }
  }
  if (a.status) {
    if (odd) atomicOr(a.status, kStatusBadLength);
    if (lost) atomicOr(a.status, kStatusBadSlot);
  }
}

namespace {
template <int D>
int run_accept(const Kv4AcceptArgs& a, cudaStream_t stream) {
  const void* fn = reinterpret_cast<const void*>(lora_kv4_accept_kernel<D>);
  const size_t smem = a.max_path <= kAcceptOnce ? 0 : a.max_path * Kv4Entry<D>::kLanes * sizeof(Kv4Entry<D>);
  if (ensure_smem_attr(fn, smem) != 0) return -6;
  const int warps = std::min(kAcceptWarps, a.num_kv_heads);
  Kv4AcceptArgs p = a;
  return launch_pdl(fn, dim3(a.num_seqs, (a.num_kv_heads + warps - 1) / warps), dim3(warps * 32), smem, stream, 0,
                    &p);
}
}  // namespace

int launch_kv4_accept(const Kv4AcceptArgs& a, cudaStream_t stream) {
  return a.head_dim == 128 ? run_accept<128>(a, stream) : run_accept<64>(a, stream);
}

}  // namespace grg
