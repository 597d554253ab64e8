// Eviction from the 4-bit cache by accumulated attention weight.  Of a sequence's n keys in one
// head, `budget` stay: the protected ones (positions below sink, the newest `recent`), then
// those of the largest weight, ties to the lowest index; the kept keys from `budget` on take
// the places of the others below it, the first the first, with their weights and positions.
//
// One CTA has a head of a sequence.  A key's rank is that of a 32-bit integer that orders like
// its weight (protected keys above all, NaN below), so the budget-th largest is found by
// counting digits of 11, 11 and 10 bits from the top (a radix selection).  Then each thread goes
// over a run of neighbouring keys: one sum over the threads gives holes and movers their
// numbers in the order of the indices, and D / 16 lanes move an entry.  Integers throughout:
// the result is exact and does not depend on timing.
#include <algorithm>

#include "kv4_move.cuh"
#include "launch.h"
#include "layer.h"

namespace grg {

namespace {
constexpr int kEvictBins = 2048;  // of a digit
constexpr int kEvictBatch = 8;    // keys that a thread asks for together
constexpr int kEvictMoves = 4;    // entries that a lane has in flight
// CTAs of 256 threads for up to kEvictSmall keys, of 1024 beyond.  Keys behind the last that
// shared memory holds are formed again wherever they are looked at.
constexpr int kEvictSmall = 4096;
constexpr int kEvictKeysMax = 40960;
constexpr int kEvictTable = 2048;  // pages whose numbers are kept in shared memory

template <int T>
struct EvictShared {
  static constexpr int kList = 2 * T;  // holes, and movers, listed at a time
  __align__(16) int bins[kEvictBins];
  int hole[kList], mover[kList];
  int2 warp_sum[32];
  int digit, rank, equal;  // the bin in which the rank falls, the rank within it, its keys
  int cut;
};
}  // namespace

template <int D, int T>
__global__ void __launch_bounds__(T, T == 256 ? 4 : 1)
    lora_kv4_evict_kernel(const __grid_constant__ Kv4EvictArgs a) {
  using Entry = Kv4Entry<D>;
  using Shared = EvictShared<T>;
  constexpr int LANES = Entry::kLanes, WARPS = T / 32;
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  int32_t* s_table = reinterpret_cast<int32_t*>(smem + sizeof(Shared));
  uint32_t* s_keys = reinterpret_cast<uint32_t*>(s_table + a.smem_pages);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / a.num_kv_heads, h = blockIdx.x - b * a.num_kv_heads;
  for (int i = tid; i < kEvictBins / 4; i += T) reinterpret_cast<int4*>(sh.bins)[i] = make_int4(0, 0, 0, 0);
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
    for (int j0 = tid; j0 < n; j0 += T * kEvictBatch) {
      int held[kEvictBatch];
#pragma unroll
      for (int u = 0; u < kEvictBatch; ++u) held[u] = j0 + u * T < n ? key_pos[j0 + u * T] : 0;
#pragma unroll
      for (int u = 0; u < kEvictBatch; ++u)
        if (held[u] < 0) key_pos[j0 + u * T] = position(j0 + u * T, -1);
    }
    return;
  }

  // ---- the keys' integers, and how often each first digit comes
  const long long newest = static_cast<long long>(last) - a.recent;  // positions above are protected
  auto rank_key = [&](float w, int pos) -> uint32_t {
    if (pos < a.sink || pos > newest) return 0xFFFFFFFFu;
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);  // (-0 as 0)
    return u >> 31 ? ~u : u | 0x80000000u;
  };
  const int32_t* table = a.page_table + b * a.table_stride;
  for (int i = tid; i < min((n + a.page_size - 1) / a.page_size, a.smem_pages); i += T) s_table[i] = __ldg(table + i);
  __syncthreads();
  for (int j0 = tid; j0 < n; j0 += T * kEvictBatch) {
    int held[kEvictBatch];
    float w[kEvictBatch];
#pragma unroll
    for (int u = 0; u < kEvictBatch; ++u) {
      const bool in = j0 + u * T < n;
      held[u] = in ? key_pos[j0 + u * T] : 0;
      w[u] = in ? weights[j0 + u * T] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kEvictBatch; ++u) {
      const int j = j0 + u * T;
      if (j < n) {
        const int pos = position(j, held[u]);
        const uint32_t key = rank_key(w[u], pos);
        if (j < a.smem_keys) s_keys[j] = key;
        if (held[u] < 0 && j < budget) key_pos[j] = pos;
        atomicAdd(&sh.bins[key >> 21], 1);
      }
    }
  }
  __syncthreads();
  auto key_of = [&](int j) -> uint32_t {
    return j < a.smem_keys ? s_keys[j] : rank_key(weights[j], position(j, key_pos[j]));
  };

  // Sums over the threads in front of this one, and over all, of two counts.
  auto sums = [&](int2 mine, int2& all) {
    int2 run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, run.x, o), y = __shfl_up_sync(0xffffffffu, run.y, o);
      if (lane >= o) run.x += x, run.y += y;
    }
    if (lane == 31) sh.warp_sum[warp] = run;
    __syncthreads();
    const int2 w = lane < WARPS ? sh.warp_sum[lane] : make_int2(0, 0);
    int2 to = w;
#pragma unroll
    for (int o = 1; o < WARPS; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, to.x, o), y = __shfl_up_sync(0xffffffffu, to.y, o);
      if (lane >= o) to.x += x, to.y += y;
    }
    all = make_int2(__shfl_sync(0xffffffffu, to.x, WARPS - 1), __shfl_sync(0xffffffffu, to.y, WARPS - 1));
    return make_int2(__shfl_sync(0xffffffffu, to.x - w.x, warp) + run.x - mine.x,
                     __shfl_sync(0xffffffffu, to.y - w.y, warp) + run.y - mine.y);
  };

  // ---- the budget-th largest: its digits from the top, until all keys with those stay
  uint32_t least = 0;  // the digits so far; in the end, the least that stays
  int rank = budget, equal = 0;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    constexpr int kBinsOf[3] = {2048, 2048, 1024};
    const int bins = kBinsOf[pass];
    if (pass > 0) {
      const int above = pass == 1 ? 21 : 10;
      for (int j0 = tid; j0 < n; j0 += T * kEvictBatch) {
        uint32_t key[kEvictBatch];
#pragma unroll
        for (int u = 0; u < kEvictBatch; ++u) key[u] = j0 + u * T < n ? key_of(j0 + u * T) : ~least;
#pragma unroll
        for (int u = 0; u < kEvictBatch; ++u)
          if (key[u] >> above == least >> above) atomicAdd(&sh.bins[(key[u] >> shift) & (bins - 1)], 1);
      }
      __syncthreads();
    }
    // each thread has a run of bins, from the top, which it leaves empty
    constexpr int PER = kEvictBins / T;  // 8 or 2
    int c[PER], sum = 0;
    int* own = sh.bins + bins - PER - tid * PER;
    const bool has = tid * PER < bins;
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
      const int2 x = has ? *reinterpret_cast<const int2*>(own + PER - 2 - i) : make_int2(0, 0);
      c[i] = x.y, c[i + 1] = x.x;
      if (has) *reinterpret_cast<int2*>(own + PER - 2 - i) = make_int2(0, 0);
      sum += x.x + x.y;
    }
    int2 all;
    int seen = sums(make_int2(sum, 0), all).x;
    if (seen < rank && rank <= seen + sum) {  // one thread's
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (seen < rank && rank <= seen + c[i])
          sh.digit = bins - 1 - (tid * PER + i), sh.rank = rank - seen, sh.equal = c[i];
        seen += c[i];
      }
    }
    __syncthreads();
    least |= static_cast<uint32_t>(sh.digit) << shift;
    rank = sh.rank, equal = sh.equal;
    if (rank == equal) break;
  }

  // ---- where only some of the keys equal to it stay, the last index that does
  // (a thread's run of keys: of odd length, so that a warp's reads are in different banks)
  int cut = n;
  if (rank < equal) {
    const int run = (n / T + 1) | 1, j0 = min(tid * run, n), j1 = j0 + min(run, n - j0);
    int count = 0;
#pragma unroll 8
    for (int j = j0; j < j1; ++j) count += key_of(j) == least ? 1 : 0;
    int2 all;
    int seen = sums(make_int2(count, 0), all).x;
    if (seen < rank && rank <= seen + count)
      for (int j = j0; j < j1; ++j)
        if (key_of(j) == least && ++seen == rank) {
          sh.cut = j;
          break;
        }
    __syncthreads();
    cut = sh.cut;
  }
  auto stays = [&](int j) {
    const uint32_t key = key_of(j);
    return key > least || (key == least && j <= cut);
  };
  // Of up to 32 keys from j on, those that stay, as bits.
  auto staying = [&](int j, int count) {
    uint32_t bits = 0;
#pragma unroll 8
    for (int i = 0; i < count; ++i) bits |= (stays(j + i) ? 1u : 0u) << i;
    return bits;
  };

  // ---- holes below the budget, movers from it on: as many of the one as of the other
  const int hrun = (budget / T + 1) | 1, h0 = min(tid * hrun, budget), h1 = h0 + min(hrun, budget - h0);
  const int mrun = ((n - budget) / T + 1) | 1;
  const int m0 = budget + min(tid * mrun, n - budget), m1 = m0 + min(mrun, n - m0);
  int2 count = make_int2(0, 0), all;
  uint32_t hole_bits = 0, mover_bits = 0;  // those of the first 32 keys of a run
  for (int j = h0; j < h1; j += 32) {
    const int some = min(h1 - j, 32);
    const uint32_t bits = staying(j, some) ^ (some == 32 ? ~0u : (1u << some) - 1u);
    if (j == h0) hole_bits = bits;
    count.x += __popc(bits);
  }
  for (int j = m0; j < m1; j += 32) {
    const uint32_t bits = staying(j, min(m1 - j, 32));
    if (j == m0) mover_bits = bits;
    count.y += __popc(bits);
  }
  const int2 first = sums(count, all);

  const Kv4Pages pages{a.cache, table, a.num_pages, a.num_kv_heads, a.page_size};
  auto block_of = [&](int j) {
    const int pg = j / a.page_size;
    return pages.block_of_page<D>(pg < a.smem_pages ? s_table[pg] : __ldg(table + pg), j - pg * a.page_size, h);
  };
  bool lost = false;
  // where this thread's lists go on: the 32 keys' bits that are left, their first key, the next number
  int hole_j = h0, hole_i = first.x, mover_j = m0, mover_i = first.y;
  for (int from = 0; from < all.x; from += Shared::kList) {  // the moves [from, from + kList)
    const int to = min(from + Shared::kList, all.x);
    while (hole_i < to && hole_j < h1) {
      if (hole_bits == 0) {
        hole_j += 32;
        if (hole_j < h1) {
          const int some = min(h1 - hole_j, 32);
          hole_bits = staying(hole_j, some) ^ (some == 32 ? ~0u : (1u << some) - 1u);
        }
        continue;
      }
      sh.hole[hole_i++ - from] = hole_j + __ffs(hole_bits) - 1;
      hole_bits &= hole_bits - 1;
    }
    while (mover_i < to && mover_j < m1) {
      if (mover_bits == 0) {
        mover_j += 32;
        if (mover_j < m1) mover_bits = staying(mover_j, min(m1 - mover_j, 32));
        continue;
      }
      sh.mover[mover_i++ - from] = mover_j + __ffs(mover_bits) - 1;
      mover_bits &= mover_bits - 1;
    }
    __syncthreads();
    constexpr int EACH = T / LANES;
    const int part = tid % LANES;
    for (int i0 = tid / LANES; i0 < to - from; i0 += kEvictMoves * EACH) {
      Entry e[kEvictMoves];
      uint32_t state[kEvictMoves];  // lane 0: the weight, lane 1: the position
      uint8_t* source[kEvictMoves];
      int j[kEvictMoves];
#pragma unroll
      for (int u = 0; u < kEvictMoves; ++u) {
        j[u] = sh.mover[min(i0 + u * EACH, to - from - 1)];
        source[u] = block_of(j[u]);
      }
#pragma unroll
      for (int u = 0; u < kEvictMoves; ++u) {
        if (source[u]) e[u].load(source[u], j[u] % 16, part);
        if (part < 2)
          asm volatile("ld.global.u32 %0, [%1];\n" : "=r"(state[u])
                       : "l"(part == 0 ? static_cast<const void*>(weights + j[u]) : static_cast<const void*>(key_pos + j[u])));
      }
#pragma unroll
      for (int u = 0; u < kEvictMoves; ++u) {
        const int i = i0 + u * EACH;
        if (i < to - from) {
          const int to_j = sh.hole[i];
          uint8_t* target = block_of(to_j);
          if (source[u] && target) e[u].store(target, to_j % 16, part);
          else lost = true;
          if (part == 0) weights[to_j] = __uint_as_float(state[u]);
          if (part == 1) key_pos[to_j] = position(j[u], static_cast<int>(state[u]));
        }
      }
    }
    __syncthreads();
  }
  for (int j = budget + tid; j < n; j += T) key_pos[j] = -1;
  if (lost && a.status) atomicOr(a.status, kStatusBadSlot);
}

namespace {
template <int D, int T>
int run_evict(const Kv4EvictArgs& a, cudaStream_t stream) {
  const void* fn = reinterpret_cast<const void*>(lora_kv4_evict_kernel<D, T>);
  const size_t smem = sizeof(EvictShared<T>) + (static_cast<size_t>(a.smem_keys) + a.smem_pages) * 4;
  if (ensure_smem_attr(fn, smem) != 0) return -6;
  Kv4EvictArgs p = a;
  return launch_pdl(fn, dim3(a.num_seqs * a.num_kv_heads), dim3(T), smem, stream, 0, &p);
}
}  // namespace

int launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t stream) {
  Kv4EvictArgs p = a;
  const int most = static_cast<int>(std::min<long long>(a.capacity, a.table_stride * a.page_size));
  p.smem_keys = std::min(most, kEvictKeysMax);
  p.smem_pages = std::min((most + a.page_size - 1) / a.page_size, kEvictTable);
  if (most <= kEvictSmall)
    return a.head_dim == 128 ? run_evict<128, 256>(p, stream) : run_evict<64, 256>(p, stream);
  return a.head_dim == 128 ? run_evict<128, 1024>(p, stream) : run_evict<64, 1024>(p, stream);
}

}  // namespace grg
