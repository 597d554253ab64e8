// Eviction from the 4-bit cache by accumulated attention weight.  Of a sequence's n keys in one
// head, `budget` stay: the protected ones (positions below sink, the newest `recent`), then
// those of the largest weight, ties to the lowest index; the kept keys from `budget` on take
// the places of the others below it, the first the first, with their weights and positions.
//
// One CTA has a head of a sequence.  A key's rank is that of a 32-bit integer that orders like
// its weight (protected keys above all, NaN below), so the budget-th largest is found by
// counting digits of 11, 11 and 10 bits from the top (a radix selection); a scan in the
// order of the indices lists holes and movers, a stretch at a time, and D / 16 lanes move an
// entry.  Integers throughout: the result is exact and does not depend on timing.
#include <algorithm>

#include "kv4_move.cuh"
#include "launch.h"
#include "layer.h"

namespace grg {

namespace {
constexpr int kEvictMaxThreads = 1024;
constexpr int kEvictBins = 2048;       // of a digit
constexpr int kEvictRing = 2048;       // holes (and movers) listed ahead
constexpr int kEvictKeysMax = 12288;   // keys whose integers are kept in shared memory
constexpr int kEvictUnroll = 4;        // entries in flight per lane

struct EvictShared {
  uint32_t bins[kEvictBins];
  int hole[kEvictRing], mover[kEvictRing];
  int count[2][32];       // a scan's warps
  int warp_sum[32];
  uint32_t digit;         // the bin in which the rank falls
  int rank, equal;        // the rank within it, and its keys
  int cut;
};
}  // namespace

template <int D>
__global__ void __launch_bounds__(kEvictMaxThreads)
    lora_kv4_evict_kernel(const __grid_constant__ Kv4EvictArgs a) {
  using Entry = Kv4Entry<D>;
  constexpr int LANES = Entry::kLanes;
  extern __shared__ __align__(16) unsigned char smem[];
  EvictShared& sh = *reinterpret_cast<EvictShared*>(smem);
  uint32_t* s_keys = reinterpret_cast<uint32_t*>(smem + sizeof(EvictShared));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x, warps = T >> 5;
  const int b = blockIdx.x / a.num_kv_heads, h = blockIdx.x - b * a.num_kv_heads;
  pdl_wait();
  pdl_launch_dependents();

  const int n0 = a.kv_len[b], last = a.last_pos[b];
  const long long room = min(a.table_stride * a.page_size, static_cast<long long>(a.capacity));
  const int n = static_cast<int>(min(static_cast<long long>(max(n0, 0)), room));
  const int budget = a.budget;
  if (tid == 0 && h == 0) {
    a.kv_len_out[b] = min(n, budget);
    if (n != n0 && a.status) atomicOr(a.status, kStatusBadLength);
  }
  float* weights = a.weights + (static_cast<long long>(b) * a.num_kv_heads + h) * a.capacity;
  int32_t* key_pos = a.key_pos + (static_cast<long long>(b) * a.num_kv_heads + h) * a.capacity;
  auto position = [&](int j, int held) {  // a key without a position was appended since the last eviction
    return held < 0 ? static_cast<int>(last - (static_cast<long long>(n) - 1 - j)) : held;
  };
  if (n <= budget) {
    for (int j = tid; j < n; j += T)
      if (key_pos[j] < 0) key_pos[j] = position(j, -1);
    return;
  }

  // ---- the keys' integers
  const long long newest = static_cast<long long>(last) - a.recent;  // positions above are protected
  auto rank_key = [&](float w, int pos) -> uint32_t {
    if (pos < a.sink || pos > newest) return 0xFFFFFFFFu;
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);  // (-0 as 0)
    return u >> 31 ? ~u : u | 0x80000000u;
  };
  auto key_of = [&](int j) -> uint32_t {
    return j < a.smem_keys ? s_keys[j] : rank_key(weights[j], position(j, key_pos[j]));
  };
  for (int i = tid; i < kEvictBins; i += T) sh.bins[i] = 0;
  __syncthreads();
  for (int j = tid; j < n; j += T) {
    const int held = key_pos[j], pos = position(j, held);
    const uint32_t key = rank_key(weights[j], pos);
    if (j < a.smem_keys) s_keys[j] = key;
    if (held < 0 && j < budget) key_pos[j] = pos;
    atomicAdd(&sh.bins[key >> 21], 1u);
  }

  // ---- the budget-th largest: its digits from the top
  uint32_t prefix = 0;  // the digits so far
  int rank = budget, equal = 0;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bins = pass == 2 ? 1024 : 2048;
    if (pass > 0) {
      const int above = pass == 1 ? 21 : 10;
      for (int i = tid; i < bins; i += T) sh.bins[i] = 0;
      __syncthreads();
      for (int j = tid; j < n; j += T) {
        const uint32_t key = key_of(j);
        if (key >> above == prefix >> above) atomicAdd(&sh.bins[(key >> shift) & (bins - 1)], 1u);
      }
    }
    __syncthreads();
    // each thread has a run of bins, from the top; a scan over the threads' sums
    const int per = bins / min(T, bins);
    int sum = 0;
    if (tid * per < bins)
      for (int i = 0; i < per; ++i) sum += sh.bins[bins - 1 - (tid * per + i)];
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    if (lane == 31) sh.warp_sum[warp] = run;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
    before += run - sum;
    if (before < rank && rank <= before + sum) {  // one thread's
      int seen = before;
      for (int i = 0; i < per; ++i) {
        const int bin = bins - 1 - (tid * per + i), c = sh.bins[bin];
        if (rank <= seen + c) {
          sh.digit = bin, sh.rank = rank - seen, sh.equal = c;
          break;
        }
        seen += c;
      }
    }
    __syncthreads();
    prefix |= sh.digit << shift;
    rank = sh.rank, equal = sh.equal;
    __syncthreads();
  }

  // ---- where only some of the keys equal to it stay, the last index that does
  // A scan in the order of the indices: the flagged ones before this thread's in the tile,
  // and of the whole tile.
  int turn = 0;
  auto scan = [&](bool flag, int& total) {
    const uint32_t votes = __ballot_sync(0xffffffffu, flag);
    if (lane == 0) sh.count[turn][warp] = __popc(votes);
    __syncthreads();
    int c = lane < warps ? sh.count[turn][lane] : 0;
    int run = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    total = __shfl_sync(0xffffffffu, run, 31);
    turn ^= 1;
    return __shfl_sync(0xffffffffu, run - c, warp) + __popc(votes & ((1u << lane) - 1u));
  };
  int cut = n;
  if (rank < equal) {
    int found = 0;
    for (int j0 = 0;; j0 += T) {
      int total;
      const bool is = j0 + tid < n && key_of(j0 + tid) == prefix;
      const int at = found + scan(is, total);
      if (is && at == rank - 1) sh.cut = j0 + tid;
      found += total;
      if (found >= rank) break;
    }
    __syncthreads();
    cut = sh.cut;
  }
  auto stays = [&](int j) {
    const uint32_t key = key_of(j);
    return key > prefix || (key == prefix && j <= cut);
  };

  // ---- holes below the budget, movers from it on, and the moves
  const Kv4Pages pages{a.cache, a.page_table + b * a.table_stride, a.num_pages, a.num_kv_heads, a.page_size};
  int holes = 0, movers = 0, moved = 0;
  int next_hole = 0, next_mover = budget;
  bool lost = false;
  while (next_hole < budget || next_mover < n) {
    while (next_hole < budget && holes + T - moved <= kEvictRing) {
      int total;
      const int j = next_hole + tid;
      const bool is = j < budget && !stays(j);
      const int at = holes + scan(is, total);
      if (is) sh.hole[at % kEvictRing] = j;
      holes += total, next_hole += T;
    }
    while (next_mover < n && movers + T - moved <= kEvictRing) {
      int total;
      const int j = next_mover + tid;
      const bool is = j < n && stays(j);
      const int at = movers + scan(is, total);
      if (is) sh.mover[at % kEvictRing] = j;
      movers += total, next_mover += T;
    }
    __syncthreads();
    const int to_move = min(holes, movers);
    const int part = tid % LANES, each = T / LANES;
    for (int i0 = moved + tid / LANES; i0 < to_move; i0 += kEvictUnroll * each) {
      Entry e[kEvictUnroll];
      float w[kEvictUnroll];
      int pos[kEvictUnroll];
      bool got[kEvictUnroll];
#pragma unroll
      for (int u = 0; u < kEvictUnroll; ++u) {
        const int i = i0 + u * each;
        got[u] = false;
        if (i < to_move) {
          const int from = sh.mover[i % kEvictRing];
          const uint8_t* block = pages.block<D>(from, h);
          got[u] = block != nullptr;
          if (block) e[u].load(block, from % 16, part);
          if (part == 0) w[u] = weights[from];
          if (part == 1) pos[u] = position(from, key_pos[from]);
        }
      }
#pragma unroll
      for (int u = 0; u < kEvictUnroll; ++u) {
        const int i = i0 + u * each;
        if (i < to_move) {
          const int to = sh.hole[i % kEvictRing];
          uint8_t* block = pages.block<D>(to, h);
          if (got[u] && block) e[u].store(block, to % 16, part);
          else lost = true;
          if (part == 0) weights[to] = w[u];
          if (part == 1) key_pos[to] = pos[u];
        }
      }
    }
    moved = to_move;
    __syncthreads();
  }
  for (int j = budget + tid; j < n; j += T) key_pos[j] = -1;
  if (lost && a.status) atomicOr(a.status, kStatusBadSlot);
}

int launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t stream) {
  const void* fn = a.head_dim == 128 ? reinterpret_cast<const void*>(lora_kv4_evict_kernel<128>)
                                     : reinterpret_cast<const void*>(lora_kv4_evict_kernel<64>);
  Kv4EvictArgs p = a;
  const int most = static_cast<int>(std::min<long long>(a.capacity, a.table_stride * a.page_size));
  p.smem_keys = std::min(most, kEvictKeysMax);
  const size_t smem = sizeof(EvictShared) + static_cast<size_t>(p.smem_keys) * 4;
  if (ensure_smem_attr(fn, smem) != 0) return -6;
  const int threads = most > 4096 ? kEvictMaxThreads : 256;
  return launch_pdl(fn, dim3(a.num_seqs * a.num_kv_heads), dim3(threads), smem, stream, 0, &p);
}

}  // namespace grg
