// Eviction from the 4-bit cache by accumulated attention weight.  Of a sequence's n keys in one
// head, `budget` stay: the protected ones (positions below sink, the newest `recent`), then
// those of the largest weight, ties to the lowest index; the kept keys from `budget` on take
// the places of the others below it, the first the first, with their weights and positions.
//
// A key's rank is that of a 32-bit integer that orders like its weight (protected keys above
// all, NaN below).  Then each thread goes over a run of neighbouring keys: one sum over the
// threads gives holes and movers their numbers in the order of the indices, and D / 16 lanes
// move an entry.  Integers throughout: the result is exact and does not depend on timing.
//
// The budget-th largest is found by counting digits of 11, 11 and 10 bits from the top (a radix
// selection), until all keys with the digits so far stay.  A CTA has a head; where heads are few and
// many keys may move, a cluster of CTAs has it: all select, each moves a part.  Integers past what
// shared memory holds are formed again wherever they are looked at.
//
// What bounds it: steps that follow one another, each with a barrier or a trip to memory (the
// weights, three counts, two sums, rounds of moves), and instructions where heads are many, not
// bytes: 2048 heads of 2000 to 2100 keys, budget 2048, take 34 us, where reading weights and
// positions once would take 5 (19.0 million warp instructions, 59 % of the issue slots); 48 heads of
// 10000 to 30000 keys, budget 2000, 38 us.  Hence the threads of a CTA: many where a head has an SM to
// itself, few where other heads fill the waits.
#include <algorithm>
#include <type_traits>

#include "kv4_move.cuh"
#include "launch.h"
#include "layer.h"

namespace grg {

namespace {
constexpr int kEvictBins = 2048;  // of a digit
constexpr int kEvictMoves = 2;    // entries that a lane has in flight (4: 42.5 us for 6 prompts, 37.7 with 2)
constexpr int kEvictShort = 2048;  // keys of a head
constexpr int kEvictLong = 16384;
constexpr int kEvictCluster = 512;  // keys that move
constexpr int kEvictKeysMax = 40960;
constexpr int kEvictTable = 2560;  // pages whose numbers are kept in shared memory

template <int T>
struct EvictShared {
  static constexpr int kList = 2 * T;  // holes, and movers, listed at a time
  __align__(16) int bins[kEvictBins];
  int hole[kList], mover[kList];
  int warp_sum[2][32];
  int digit, rank, equal;  // the bin in which the rank falls, the rank within it, its keys
  int cut;
};
}  // namespace

// ALL: shared memory holds all keys and pages.
template <int D, int T, bool ALL>
__global__ void __launch_bounds__(T, T == 256 ? 6 : T == 512 ? 3 : 1)
    lora_kv4_evict_kernel(const __grid_constant__ Kv4EvictArgs a) {
  using Entry = Kv4Entry<D>;
  using Shared = EvictShared<T>;
  constexpr int LANES = Entry::kLanes, WARPS = T / 32;
  constexpr int KEYS = 8;  // keys that a thread asks for together
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  int32_t* s_table = reinterpret_cast<int32_t*>(smem + sizeof(Shared));
  uint32_t* s_keys = reinterpret_cast<uint32_t*>(s_table + a.smem_pages);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item = blockIdx.x / a.cluster, rank_in = blockIdx.x - item * a.cluster;
  const int b = item / a.num_kv_heads, h = item - b * a.num_kv_heads;
  for (int i = tid; i < kEvictBins / 4; i += T) reinterpret_cast<int4*>(sh.bins)[i] = make_int4(0, 0, 0, 0);
  pdl_wait();
  pdl_launch_dependents();

  const int n0 = a.kv_len[b], last = a.last_pos[b];
  const long long room = min(a.table_stride * a.page_size, static_cast<long long>(a.capacity));
  const int n = static_cast<int>(min(static_cast<long long>(max(n0, 0)), room));
  const int budget = a.budget;
  if (tid == 0 && h == 0 && rank_in == 0) {
    a.kv_len_out[b] = min(n, budget);
    if (n != n0 && a.status) atomicOr(a.status, kStatusBadLength);
  }
  float* weights = a.weights + (static_cast<long long>(b) * a.num_kv_heads + h) * a.capacity;
  int32_t* key_pos = a.key_pos + (static_cast<long long>(b) * a.num_kv_heads + h) * a.capacity;
  const int32_t* table = a.page_table + b * a.table_stride;
  auto position = [&](int j, int held) {  // a key without a position was appended since the last eviction
    return held < 0 ? static_cast<int>(static_cast<uint32_t>(last) - static_cast<uint32_t>(n - 1 - j)) : held;
  };
  const bool over = n > budget;
  if (over)
    for (int i = tid; i < min((n + a.page_size - 1) / a.page_size, a.smem_pages); i += T) s_table[i] = __ldg(table + i);

  // ---- the keys' integers (of a sequence over its budget), new keys' positions
  // positions above are protected (where none reach, down to the least, so are all but that one: a
  // position there was never given)
  const int newest = static_cast<int>(max(static_cast<long long>(last) - a.recent, -(1ll << 31)));
  auto rank_key = [&](float w, int pos) -> uint32_t {
    if (pos < a.sink || pos > newest) return 0xFFFFFFFFu;
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);  // (-0 as 0)
    return u >> 31 ? ~u : u | 0x80000000u;
  };
  __syncthreads();  // the bins are empty
  for (int j0 = tid; j0 < n; j0 += T * KEYS) {
    int held[KEYS];
    float w[KEYS];
#pragma unroll
    for (int u = 0; u < KEYS; ++u) {
      const bool in = j0 + u * T < n;
      held[u] = in ? key_pos[j0 + u * T] : 0;
      w[u] = in && over ? weights[j0 + u * T] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < KEYS; ++u) {
      const int j = j0 + u * T;
      if (j < n) {
        const int pos = position(j, held[u]);
        if (held[u] < 0 && j < budget && rank_in == 0) key_pos[j] = pos;
        const uint32_t key = rank_key(w[u], pos);
        if (ALL || j < a.smem_keys) s_keys[j] = key;
        if (over) atomicAdd(&sh.bins[key >> 21], 1);
      }
    }
  }
  if (!over) return;
  if (a.cluster > 1) cluster_sync_all();  // (and a barrier) before any of the CTAs moves something
  else __syncthreads();
  auto key_of = [&](int j) -> uint32_t {
    if (ALL || j < a.smem_keys) return s_keys[j];
    return rank_key(weights[j], position(j, key_pos[j]));
  };

  // The sum over the threads in front of this one, and over all.
  auto sums = [&](int mine, int& all, int* turn) {
    int run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += x;
    }
    if (lane == 31) turn[warp] = run;
    __syncthreads();
    const int w = lane < WARPS ? turn[lane] : 0;
    all = __reduce_add_sync(0xffffffffu, w);
    return __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + run - mine;
  };

  // ---- the budget-th largest, or a bound below it with as many keys
  uint32_t least = 0;
  int rank = budget, equal = 0;  // of the keys equal to it, how many stay, and how many there are
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {  // digits of 11, 11 and 10 bits
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    if (pass > 0) {
      const int above = pass == 1 ? 21 : 10;
#pragma unroll 4
      for (int j = tid; j < n; j += T) {
        const uint32_t k = key_of(j);
        if (k >> above == least >> above) atomicAdd(&sh.bins[(k >> shift) & (bins - 1)], 1);
      }
      __syncthreads();
    }
    // each thread has a run of bins, from the top, which it leaves empty
    constexpr int PER = kEvictBins / T;  // 8 or 2
    int2 c[PER / 2];
    int sum = 0;
    int2* own = reinterpret_cast<int2*>(sh.bins + bins - PER - tid * PER);
    const bool has = tid * PER < bins;
#pragma unroll
    for (int i = 0; i < PER / 2; ++i) {
      c[i] = has ? own[PER / 2 - 1 - i] : make_int2(0, 0);
      if (has) own[PER / 2 - 1 - i] = make_int2(0, 0);
      sum += c[i].x + c[i].y;
    }
    int all;
    int seen = sums(sum, all, sh.warp_sum[0]);
    if (seen < rank && rank <= seen + sum) {  // one thread's
#pragma unroll
      for (int i = 0; i < PER / 2; ++i) {
        if (seen < rank && rank <= seen + c[i].x + c[i].y) {
          const bool second = rank > seen + c[i].y;
          sh.digit = bins - 1 - tid * PER - 2 * i - (second ? 1 : 0);
          sh.rank = rank - seen - (second ? c[i].y : 0), sh.equal = second ? c[i].x : c[i].y;
        }
        seen += c[i].x + c[i].y;
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
#pragma unroll 4
    for (int j = j0; j < j1; ++j) count += key_of(j) == least ? 1 : 0;
    int all;
    int seen = sums(count, all, sh.warp_sum[0]);
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
#pragma unroll 4
    for (int i = 0; i < count; ++i) bits |= (stays(j + i) ? 1u : 0u) << i;
    return bits;
  };

  // ---- holes below the budget, movers from it on: as many of the one as of the other
  const int hrun = (budget / T + 1) | 1, h0 = min(tid * hrun, budget), h1 = h0 + min(hrun, budget - h0);
  const int mrun = ((n - budget) / T + 1) | 1;
  const int m0 = budget + min(tid * mrun, n - budget), m1 = m0 + min(mrun, n - m0);
  int holes = 0, movers = 0, all;
  uint32_t hole_bits = 0, mover_bits = 0;  // those of the first 32 keys of a run
  for (int j = h0; j < h1; j += 32) {
    const int some = min(h1 - j, 32);
    const uint32_t bits = staying(j, some) ^ (some == 32 ? ~0u : (1u << some) - 1u);
    if (j == h0) hole_bits = bits;
    holes += __popc(bits);
  }
  for (int j = m0; j < m1; j += 32) {
    const uint32_t bits = staying(j, min(m1 - j, 32));
    if (j == m0) mover_bits = bits;
    movers += __popc(bits);
  }
  const int first_mover = sums(movers, all, sh.warp_sum[1]), first_hole = sums(holes, all, sh.warp_sum[0]);

  const Kv4Pages pages{a.cache, table, a.num_pages, a.num_kv_heads, a.page_size};
  auto block_of = [&](int j) {
    const int pg = static_cast<int>((static_cast<unsigned long long>(j >> 4) * a.page_magic) >> 36);
    return pages.block_of_page<D>(ALL || pg < a.smem_pages ? s_table[pg] : __ldg(table + pg), j - pg * a.page_size, h);
  };
  bool lost = false;
  // this CTA's share of the moves
  const int share = (all + a.cluster - 1) / a.cluster, share0 = min(rank_in * share, all);
  const int share1 = min(share0 + share, all);
  // where this thread's lists go on: the 32 keys' bits that are left, their first key, the next number
  int hole_j = h0, hole_i = first_hole, mover_j = m0, mover_i = first_mover;
  for (int from = share0; from < share1; from += Shared::kList) {  // the moves [from, from + kList)
    const int to = min(from + Shared::kList, share1);
    while (hole_i < to && hole_j < h1) {
      if (hole_bits == 0) {
        hole_j += 32;
        if (hole_j < h1) {
          const int some = min(h1 - hole_j, 32);
          hole_bits = staying(hole_j, some) ^ (some == 32 ? ~0u : (1u << some) - 1u);
        }
        continue;
      }
      if (hole_i >= from) sh.hole[hole_i - from] = hole_j + __ffs(hole_bits) - 1;
      ++hole_i;
      hole_bits &= hole_bits - 1;
    }
    while (mover_i < to && mover_j < m1) {
      if (mover_bits == 0) {
        mover_j += 32;
        if (mover_j < m1) mover_bits = staying(mover_j, min(m1 - mover_j, 32));
        continue;
      }
      if (mover_i >= from) sh.mover[mover_i - from] = mover_j + __ffs(mover_bits) - 1;
      ++mover_i;
      mover_bits &= mover_bits - 1;
    }
    __syncthreads();
    constexpr int EACH = T / LANES;
    const int part = tid % LANES;
    auto move = [&](auto several, int i0) {  // that many entries in flight per lane
      constexpr int MOVES = decltype(several)::value;
      Entry e[MOVES];
      uint32_t state[MOVES];  // lane 0: the weight, lane 1: the position
      uint8_t* source[MOVES];
      int j[MOVES];
#pragma unroll
      for (int u = 0; u < MOVES; ++u) {
        j[u] = sh.mover[min(i0 + u * EACH, to - from - 1)];
        source[u] = block_of(j[u]);
      }
#pragma unroll
      for (int u = 0; u < MOVES; ++u) {
        if (source[u]) e[u].load(source[u], j[u] % 16, part);
        if (part < 2)
          asm volatile("ld.global.u32 %0, [%1];\n" : "=r"(state[u])
                       : "l"(part == 0 ? static_cast<const void*>(weights + j[u]) : static_cast<const void*>(key_pos + j[u])));
      }
#pragma unroll
      for (int u = 0; u < MOVES; ++u) {
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
    };
    for (int i0 = tid / LANES; i0 < to - from;) {
      if (to - from - i0 > EACH) {
        move(std::integral_constant<int, kEvictMoves>(), i0);
        i0 += kEvictMoves * EACH;
      } else {
        move(std::integral_constant<int, 1>(), i0);
        i0 += EACH;
      }
    }
    __syncthreads();
  }
  if (a.cluster > 1) cluster_sync_all();  // the movers' positions have been read
  for (int j = budget + rank_in * T + tid; j < n; j += T * a.cluster) key_pos[j] = -1;
  if (lost && a.status) atomicOr(a.status, kStatusBadSlot);
}

namespace {
template <int D, int T, bool ALL>
int run_evict(const Kv4EvictArgs& a, cudaStream_t stream) {
  const void* fn = reinterpret_cast<const void*>(lora_kv4_evict_kernel<D, T, ALL>);
  const size_t smem = sizeof(EvictShared<T>) + (static_cast<size_t>(a.smem_keys) + a.smem_pages) * 4;
  if (ensure_smem_attr(fn, smem) != 0) return -6;
  Kv4EvictArgs p = a;
  return launch_pdl(fn, dim3(a.num_seqs * a.num_kv_heads * a.cluster), dim3(T), smem, stream,
                    a.cluster > 1 ? a.cluster : 0, &p);
}
template <int D>
int run_evict(const Kv4EvictArgs& a, int threads, int most, cudaStream_t stream) {
  if (threads == 256) return run_evict<D, 256, true>(a, stream);
  if (threads == 512) return run_evict<D, 512, true>(a, stream);
  return most <= kEvictKeysMax ? run_evict<D, 1024, true>(a, stream) : run_evict<D, 1024, false>(a, stream);
}
}  // namespace

int launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t stream) {
  Kv4EvictArgs p = a;
  const int most = static_cast<int>(std::min<long long>(a.capacity, a.table_stride * a.page_size));
  p.smem_keys = std::min(most, kEvictKeysMax);
  p.smem_pages = std::min((most + a.page_size - 1) / a.page_size, kEvictTable);
  const int sms = device_sm_count();
  if (sms <= 0) return -6;
  const unsigned long long page_blocks = a.page_size / 16;
  p.page_magic = ((1ull << 36) + page_blocks - 1) / page_blocks;
  p.cluster = 1;
  const long long items = static_cast<long long>(a.num_seqs) * a.num_kv_heads;
  const int moves = std::min(a.budget, most - std::min(a.budget, most));  // of a head, at most
  // Measured, us by CTAs of 256 / 512 / 1024 threads (keys = budget + those that go):
  //   8 heads of 1000 + 24 keys 9.0 / 8.5 / 9.2, of 500 + 3500 17.1 / 12.1 / 11.5
  //   152 heads of 4096 + 104 17.7 / 13.0 / 11.4; 304 of them 21.2 / 16.8 / 21.3
  //   304 heads of 2000 + 6000 30.5 / 23.1 / 28.4; 608 heads of 2000 + 100 21.8 / 26.8 / 38.1
  //   608 heads of 8192 + 100 40.0 / 44.8 / 54.5; of 20000 + 200 (one or two CTAs an SM) 122 / - / 81
  // The host knows the buffers' widths, not the lengths: 2048 heads of 2100 keys (one state over
  // and over) take 31 us with a capacity of 2100, 49 us of 16384, 73 us of 16400 to 40960.
  // Clusters against none: 8 heads of 2000 + 28000 keys 22.8 (eight CTAs) and 31.7, 48 heads of
  // them 37.8 (two) and 43.8, 8 heads of 4096 + 4 11.4 and 10.1.
  int threads = 1024;
  if (most <= kEvictLong) {
    if (items > 3ll * sms) {
      threads = 256;
    } else if (items > sms || most <= kEvictShort) {
      threads = 512;
    }
  }
  // (integers that are formed again must not see another CTA's moves)
  if (threads == 1024 && moves >= kEvictCluster && most <= kEvictKeysMax)
    while (p.cluster < 8 && 2 * p.cluster * items <= sms) p.cluster *= 2;
  return a.head_dim == 128 ? run_evict<128>(p, threads, most, stream)
                           : run_evict<64>(p, threads, most, stream);
}

}  // namespace grg
