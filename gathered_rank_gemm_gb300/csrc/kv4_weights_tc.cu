// The key weights of sequences with many query rows (chunks of prefill, long paths), on the
// 5th-generation tensor cores.
//
// An item is 256 keys of one key head, as two tiles of 128, against all packed rows (row x head
// of the key head) that see one of them, 128 at a time:
//   S_t = K_t Q^T (M = 128 keys, N = rows),  w[key] += sum over rows of 2^(S c - lse log2 e)
// Keys are the lanes of TMEM, so a key's sum is one thread's: nothing is exchanged, no key's
// sum is cut, and each is formed in the rows' order.  K stays in TMEM while the rows pass by
// (from shared memory, K and the rows together take all of its bandwidth, 128 bytes a cycle:
// 172 us for 6 chunks).  It is widened to q's own 16-bit type: a code times its e4m3 scale has at
// most six significant bits, which bf16 holds too, so that q is copied as it is and c is
// the same for all rows.
//
// Warp roles (20 warps of 96 registers, one CTA per SM, persistent):
//  - warps 0-3 and 4-7: the sums of tile 0 and 1; a thread owns a key
//  - warps 8-15: widen K into TMEM; a thread has a key, its codes asked for an item ahead, its page two
//  - warp 16: issues the products; S has three places in TMEM, which the tiles take in turn
//  - warps 17-19: the rows' logarithms, and the rows of q, four tiles deep: by TMA, or, where a path
//    picks them, by copies of 16 bytes
// Work: few items a CTA (up to kTcDeal) are dealt out in rounds, those of most row tiles first, each
// round to the CTAs with the least so far; many stay in their own order and are cut into equal runs.
//
// Measured (GB300, bf16): 6 chunks of 700 to 2000 rows over 2000 to 5000 keys, 32 / 8 heads of 128:
// 149 us, 1170 TFLOP/s (0.61 of measured); one prompt of 8000 rows 225 us; 64 sequences of 16 rows over
// 2000 keys 72 us.  Bound by the sums: a row tile of two key tiles takes 1750 cycles; its products
// alone would take 1024, its 32768 exponentials another unit's 1024, and each value is read from
// TMEM, scaled and added by the same eight warps (two threads a key: 188 us).
#include <algorithm>

#include "kv4_weights.cuh"
#include "launch.h"

namespace grg {

namespace {
constexpr int kTcWarps = 20, kTcThreads = kTcWarps * 32;
constexpr int kTcCopiers = 96;  // threads that copy rows
constexpr int kTcLine = 512;    // threads that sum up the sequences
constexpr int kTcCtasMax = 160;
constexpr int kTcFixed = 2;     // what an item costs besides its row tiles, in row tiles (chunks: 0 to 5 measure the same)
constexpr int kTcKeys = 256;   // keys of an item
constexpr int kTcRows = 128;   // packed rows of a tile, at most: whole rows where 128 heads hold one
constexpr int kTcPairs = 512;  // (sequence, key tile) pairs that can be sorted
// Items a CTA up to which they are dealt: 6 chunks (7 items a CTA) 149 us dealt, 263 us in runs; one
// prompt of 8000 rows 224 and 403 us; 64 paths of 64 of 2000 to 4000 keys, all items alike, 101 and 96 us.
constexpr int kTcDeal = 16;
constexpr int kTcStages = 4;   // row tiles in shared memory
constexpr int kTcAhead = 8;    // row tiles' logarithms kept
constexpr int kTcPlaces = 3;   // of S in TMEM
constexpr float kTcLog2e = 1.4426950408889634f;

struct TcParams {
  Kv4WeightsArgs a;
  int max_packed_rows;  // sequences with no more packed rows are not this kernel's
  int tile_rows;        // packed rows of a tile
  int by_tma;           // q's rows come by TMA
  unsigned long long page_magic;  // ceil(2^36 / blocks of a page)
  unsigned long long wait_limit_ns;
  int wait_fault;
};

struct TcParamsTma {
  CUtensorMap q;  // [rows][heads][D], boxes of 64 columns of the heads of a tile's rows
  TcParams p;
};

struct TcShared {
  uint64_t q_full[kTcStages], q_empty[kTcStages];  // by row tile: the rows are there; their products are done
  uint64_t l_full[kTcAhead];                       // and their logarithms
  uint64_t k_full, k_empty;                        // by item
  uint64_t s_full[kTcPlaces], s_empty[kTcPlaces];  // by row tile and key tile
  uint64_t drain;
  __align__(16) float neg[kTcAhead][kTcRows];  // -lse log2 e of a tile's rows, -infinity: adds nothing
  __align__(16) uint32_t adds[kTcAhead][4];    // its rows that do (and what lies behind the last)
  uint32_t taddr;
  int abort;
  long long warp_sum[kTcLine / 32];
  long long prefix[kTcLine];  // pairs before a thread's sequences
  struct Pair {
    int b, kt, row0, rows, q0, q_rows, seq_rows, kv, end;
  } pair[kTcPairs];
  int sorted[kTcPairs];
  uint32_t order[kTcPairs];
  __align__(16) int load[kTcCtasMax];  // row tiles of each CTA so far, and its number in the low 8 bits
  int dealt[kTcDeal];                  // this CTA's items
};

// An item: its keys [256 kt, ...) and the packed rows [row0, row0 + rows) that see one of them.
struct TcItem {
  int b, h, kt;
  WeightSeq seq;
  int row0, rows;
};
__device__ __forceinline__ bool tc_mine(const WeightSeq& s, int group, int max_packed_rows) {
  return s.rows > 0 && static_cast<long long>(s.take) * group > max_packed_rows;
}
// Key tiles of a sequence: [first, first + count).
__device__ __forceinline__ int tc_first(const WeightSeq& s, int window) { return s.first_key(0, window) / kTcKeys; }
__device__ __forceinline__ int tc_count(const WeightSeq& s, int window) {
  return max((s.end + kTcKeys - 1) / kTcKeys - tc_first(s, window), 0);
}
template <bool PATH>
__device__ __forceinline__ void tc_rows(const WeightSeq& s, int kt, int group, int window, int& row0, int& rows) {
  const int before = s.kv - s.rows;
  const int key0 = kt * kTcKeys, key1 = min(key0 + kTcKeys, s.end) - 1;
  const int i0 = max(key0 - before, 0);
  long long i1 = s.take - 1;
  if (window > 0 && !(PATH && key1 >= before)) i1 = min(i1, static_cast<long long>(key1) + window - 1 - before);
  row0 = i0 * group;
  rows = i1 >= i0 ? static_cast<int>(i1 - i0 + 1) * group : 0;
}
__device__ __forceinline__ bool tc_elect() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// 16 consecutive 32-bit columns of this thread's TMEM lane: the load, and the wait for every
// load so far (the registers hold nothing before it).
__device__ __forceinline__ void tc_ld16_start(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tc_ld16_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[shared].
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// (s0, s1) * (c, c) + (n0, n1), and a sum, two fp32 at a time.
__device__ __forceinline__ void tc_fma2(float& x, float& y, uint32_t s0, uint32_t s1, float c, float n0,
                                        float n1) {
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 c, {%5, %6};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(x), "=f"(y)
      : "r"(s0), "r"(s1), "f"(c), "f"(n0), "f"(n1));
}
__device__ __forceinline__ void tc_add2(float& x, float& y, float a, float b) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n add.rn.f32x2 a, a, b;\n"
      " mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
}  // namespace

// PATH: the rows are those of paths, whose window hides no row's ancestors.  (Asked at run time it costs
// the other calls 2 %: 64 sequences of 36 packed rows 72.2 -> 73.6 us.)
template <int D, bool F16, bool PATH>
__global__ void __launch_bounds__(kTcThreads, 1)
    lora_kv4_weights_tc_kernel(const __grid_constant__ TcParamsTma params) {
  const TcParams& p = params.p;
  using B = Kv4Block<D>;
  constexpr int ATOMS = D / 64;                        // 128-byte atoms of a row
  constexpr uint32_t kAtom = 128 * 128;                // 128 rows of one
  constexpr uint32_t kTile = ATOMS * kAtom;            // an operand tile of 128 rows
  constexpr uint32_t kOffShared = kTcStages * kTile;
  constexpr uint32_t kColS = D;                        // TMEM columns: two tiles of K, then S
  constexpr uint32_t kIdesc = (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | (8u << 24);

  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (sbase - raw);
  TcShared& sh = *reinterpret_cast<TcShared*>(smem + kOffShared);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const Kv4WeightsArgs& a = p.a;
  const int group = a.num_q_heads / a.num_kv_heads;
  auto bar = [&](uint64_t& b) { return smem_u32(&b); };
  if (tid == 0) {
    for (int i = 0; i < kTcStages; ++i) {
      mbar_init(bar(sh.q_full[i]), (p.by_tma ? 1 : kTcCopiers) + (p.wait_fault ? 1 : 0));
      mbar_init(bar(sh.q_empty[i]), 1);
    }
    for (int i = 0; i < kTcPlaces; ++i) {
      mbar_init(bar(sh.s_full[i]), 1);
      mbar_init(bar(sh.s_empty[i]), 4);
    }
    mbar_init(bar(sh.k_full), 8);
    mbar_init(bar(sh.k_empty), 1);
    for (int i = 0; i < kTcAhead; ++i) mbar_init(bar(sh.l_full[i]), 3);
    mbar_init(bar(sh.drain), 1);
    fence_mbar_init();
    sh.abort = 0;
  }
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     smem_u32(&sh.taddr)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  const CtaAbort cta_abort{&sh.abort, p.wait_limit_ns};
  const int R = p.tile_rows;
  // what TMA never writes behind a tile's last row is read by the products all the same
  for (int i = tid; i < kTcStages * ATOMS * (kTcRows - R) * 8; i += kTcThreads) {
    const int tile = i / ((kTcRows - R) * 8), in = i % ((kTcRows - R) * 8);
    *reinterpret_cast<uint4*>(smem + tile * kAtom + R * 128 + in * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async();
  pdl_wait();
  pdl_launch_dependents();

  // ---- the pairs of sequence and key tile, and their order
  const int per_thread = (a.num_seqs + kTcLine - 1) / kTcLine;
  long long mine = 0;
  for (int i = 0; i < per_thread && tid < kTcLine; ++i) {
    const int b = tid * per_thread + i;
    if (b < a.num_seqs) {
      const WeightSeq s = WeightSeq::of(a, b);
      if (tc_mine(s, group, p.max_packed_rows)) mine += tc_count(s, a.window);
    }
  }
  long long run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += v;
  }
  if (lane == 31 && tid < kTcLine) sh.warp_sum[warp] = run;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long before = 0, pairs = 0;  // (in front of this thread's)
#pragma unroll
  for (int w = 0; w < kTcLine / 32; ++w) {
    if (w < warp) before += sh.warp_sum[w];
    pairs += sh.warp_sum[w];
  }
  if (tid < kTcLine) sh.prefix[tid] = before + run - mine;
  static_assert(4 * kTcCtasMax <= kTcThreads && kTcCtasMax % 16 == 0, "four lanes a CTA, in whole warps");
  if (tid < kTcCtasMax) sh.load[tid] = tid < static_cast<int>(gridDim.x) ? tid : 0x7fffffff;
  const long long items = pairs * a.num_kv_heads, G = gridDim.x;
  const bool sorted = pairs <= kTcPairs && items <= kTcDeal * G;
  __syncthreads();
  // The sequence of a pair, by one thread (the last prefix that is not past it).
  auto pair_of = [&](long long pr, TcItem& it) {
    int lo = 0;
#pragma unroll
    for (int step = kTcLine / 2; step; step /= 2)
      if (sh.prefix[lo + step] <= pr) lo += step;
    long long off = pr - sh.prefix[lo];
    for (it.b = lo * per_thread;; ++it.b) {
      it.seq = WeightSeq::of(a, it.b);
      const int n = tc_mine(it.seq, group, p.max_packed_rows) ? tc_count(it.seq, a.window) : 0;
      if (off < n) break;
      off -= n;
    }
    it.kt = tc_first(it.seq, a.window) + static_cast<int>(off);
    tc_rows<PATH>(it.seq, it.kt, group, a.window, it.row0, it.rows);
  };
  if (sorted) {
    TcItem it;
    it.rows = 0;
    if (tid < pairs) {
      pair_of(tid, it);
      sh.pair[tid] = {it.b, it.kt, it.row0, it.rows, it.seq.q0, it.seq.q_rows, it.seq.rows, it.seq.kv, it.seq.end};
    }
    __syncthreads();
    // a pair's place: those of more row tiles first, then in their own order (both in one number;
    // four lanes count a pair's place where there are threads for it)
    if (tid < kTcPairs)
      sh.order[tid] = tid < pairs ? static_cast<uint32_t>(min((it.rows + R - 1) / R, 1 << 21)) << 9 | (kTcPairs - 1 - tid) : 0u;
    __syncthreads();
    const int lanes = 4 * pairs <= kTcThreads ? 4 : 1, own_pair = tid / lanes;
    if (own_pair < (static_cast<int>(pairs) + 31) / 32 * 32) {  // (whole warps)
      const uint32_t own = sh.order[min(own_pair, kTcPairs - 1)];
      int place = 0;
#pragma unroll 4
      for (int i = tid & (lanes - 1); i < static_cast<int>(pairs); i += lanes) place += sh.order[i] > own ? 1 : 0;
      if (lanes == 4) {
        place += __shfl_xor_sync(0xffffffffu, place, 1);
        place += __shfl_xor_sync(0xffffffffu, place, 2);
      }
      if (own_pair < pairs && (tid & (lanes - 1)) == 0) sh.sorted[place] = own_pair;
    }
    __syncthreads();
    // Rounds: the CTA with the least so far takes the round's largest item, and so on.  (6 chunks of
    // 800 to 2000 rows: 760 items, the longest CTA has 1.05 of the mean; to and fro, 1.17.)
    for (int k = 0; k * G < items; ++k) {
      // (four lanes count a CTA's rank)
      const int cta = tid / 4;
      int rank = 0, size = 0;
      if (cta < kTcCtasMax) {
        const int own = sh.load[cta];
#pragma unroll 5
        for (int i = 4 * (tid & 3); i < kTcCtasMax; i += 16) {  // (CTAs that are not there count as full)
          const int4 x = *reinterpret_cast<const int4*>(sh.load + i);
          rank += (x.x < own ? 1 : 0) + (x.y < own ? 1 : 0) + (x.z < own ? 1 : 0) + (x.w < own ? 1 : 0);
        }
        rank += __shfl_xor_sync(0xffffffffu, rank, 1);
        rank += __shfl_xor_sync(0xffffffffu, rank, 2);
        const long long e = k * G + rank;
        const bool has = cta < G && e < items;
        if (has && (tid & 3) == 0)
          size = min((sh.pair[sh.sorted[static_cast<int>(e) / a.num_kv_heads]].rows + R - 1) / R + kTcFixed, 1 << 18);
        if ((tid & 3) == 0 && cta == blockIdx.x) sh.dealt[k] = has ? static_cast<int>(e) : -1;
      }
      __syncthreads();
      if ((tid & 3) == 0 && cta < kTcCtasMax) sh.load[cta] += size << 8;
      __syncthreads();
    }
  }
  const uint32_t taddr = sh.taddr;
  // The CTA's items one after the other; false: there is no (further) one.
  const long long per = quotient(items + G - 1, G);
  struct Walk {
    TcItem it;
    long long k;
  };
  auto deal = [&](Walk& w) -> bool {  // the item of this CTA's round k (one without is the last)
    if (w.k * G >= items) return false;
    const int e = sh.dealt[w.k];
    if (e < 0) return false;
    const auto& x = sh.pair[sh.sorted[e / a.num_kv_heads]];
    w.it.h = e % a.num_kv_heads;
    w.it.b = x.b, w.it.kt = x.kt, w.it.row0 = x.row0, w.it.rows = x.rows;
    w.it.seq.q0 = x.q0, w.it.seq.q_rows = x.q_rows, w.it.seq.rows = x.seq_rows, w.it.seq.kv = x.kv, w.it.seq.end = x.end;
    return true;
  };
  auto first_item = [&](Walk& w) -> bool {
    w.k = 0;
    if (sorted) return deal(w);
    // (own order: sequence, head, key tile; a pair stands for a key tile of one head here)
    const long long e = blockIdx.x * per;
    if (e >= items) return false;
    int lo = 0;
#pragma unroll
    for (int step = kTcLine / 2; step; step /= 2)
      if (sh.prefix[lo + step] * a.num_kv_heads <= e) lo += step;
    long long off = e - sh.prefix[lo] * a.num_kv_heads;
    int n;
    for (w.it.b = lo * per_thread;; ++w.it.b) {
      w.it.seq = WeightSeq::of(a, w.it.b);
      n = tc_mine(w.it.seq, group, p.max_packed_rows) ? tc_count(w.it.seq, a.window) : 0;
      if (off < static_cast<long long>(n) * a.num_kv_heads) break;
      off -= static_cast<long long>(n) * a.num_kv_heads;
    }
    w.it.h = static_cast<int>(quotient(off, n));
    w.it.kt = tc_first(w.it.seq, a.window) + static_cast<int>(off - static_cast<long long>(w.it.h) * n);
    tc_rows<PATH>(w.it.seq, w.it.kt, group, a.window, w.it.row0, w.it.rows);
    return true;
  };
  auto next_item = [&](Walk& w) -> bool {
    ++w.k;
    if (sorted) return deal(w);
    if (w.k >= per || blockIdx.x * per + w.k >= items) return false;
    if (++w.it.kt - tc_first(w.it.seq, a.window) == tc_count(w.it.seq, a.window)) {
      if (++w.it.h == a.num_kv_heads) {
        w.it.h = 0;
        do w.it.seq = WeightSeq::of(a, ++w.it.b);
        while (!tc_mine(w.it.seq, group, p.max_packed_rows) || tc_count(w.it.seq, a.window) == 0);
      }
      w.it.kt = tc_first(w.it.seq, a.window);
    }
    tc_rows<PATH>(w.it.seq, w.it.kt, group, a.window, w.it.row0, w.it.rows);
    return true;
  };
  auto page_of = [&](int j) {  // j / page_size, for j / 16 < 2^27 and pages of up to 64 blocks
    return static_cast<int>((static_cast<unsigned long long>(j >> 4) * p.page_magic) >> 36);
  };
  auto given_up = [&]() { return __any_sync(0xffffffffu, cta_abort.raised()) != 0; };

  if (warp < 8) {
    // -------------------------------------------------------------- sums
    const int sub = warp >> 2, key_in = sub * 128 + (warp & 3) * 32 + lane;
    const uint32_t tS = taddr + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kColS;
    const float c = score_factor(1.0f, a.score_scale * kTcLog2e);
    uint32_t t = 0;  // row tiles so far
    uint32_t place = sub, turn = 0;  // where S of (t, sub) is, and how often it was used before
    bool lost = false;
    // This thread's key of an item: what it has so far and its page are asked for an item ahead.
    struct Key {
      float* w;         // null: not this call's
      float old;
      int page;
      int row0, rows;   // the item's
      int see0, see1;   // the packed rows that see the key
    };
    auto key_of = [&](const TcItem& it) {
      Key x;
      const int j = it.kt * kTcKeys + key_in, before_rows = it.seq.kv - it.seq.rows;
      const bool there = j < it.seq.end && j >= it.seq.first_key(0, a.window);
      x.w = nullptr;
      x.old = 0.0f;
      x.page = 0;
      if (there) {
        x.w = a.weights + (static_cast<long long>(it.b) * a.num_kv_heads + it.h) * a.capacity + j;
        x.page = __ldg(a.page_table + it.b * a.table_stride + page_of(j));
        if (j < before_rows) x.old = *x.w;
      }
      x.row0 = it.row0, x.rows = it.rows;
      x.see0 = max(j - before_rows, 0) * group;
      x.see1 = it.row0 + it.rows;
      if (a.window > 0 && !(PATH && j >= before_rows)) {
        const long long i1 = static_cast<long long>(j) + a.window - before_rows;  // behind the last
        if (i1 * group < x.see1) x.see1 = static_cast<int>(max(i1 * group, 0ll));
      }
      return x;
    };
    // A wait that looks at the flag only where the phase is not over yet.
    auto over = [&](uint64_t& b, uint32_t parity) {
      return mbar_try_wait(bar(b), parity) || cta_abort.wait(bar(b), parity);
    };
    auto item_sum = [&](const Key& key) {
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      // the packed rows that all of the warp's keys see, and those that some key does
      const int all0 = __reduce_max_sync(0xffffffffu, key.see0), all1 = __reduce_min_sync(0xffffffffu, key.see1);
      const int any0 = __reduce_min_sync(0xffffffffu, key.see0), any1 = __reduce_max_sync(0xffffffffu, key.see1);
      for (int r0 = key.row0; r0 < key.row0 + key.rows; r0 += R, ++t) {
        const int slot = t % kTcAhead;
        bool ok = over(sh.l_full[slot], (t / kTcAhead) & 1);
        ok = over(sh.s_full[place], turn & 1) && ok;
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        const uint4 adds = *reinterpret_cast<const uint4*>(sh.adds[slot]);
        const bool masked = r0 < all0 || r0 + R > all1 || (adds.x & adds.y & adds.z & adds.w) != ~0u;
        const uint32_t at = tS + place * kTcRows;
        const float4* neg = reinterpret_cast<const float4*>(sh.neg[slot]);
        if (!masked) {
          uint32_t v[2][16];
          tc_ld16_start(at, v[0]);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t (&s)[16] = v[q & 1];
            tc_ld16_wait(s);
            if (q < 7) tc_ld16_start(at + 16 * (q + 1), v[(q + 1) & 1]);
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 n = neg[4 * q + e / 4];
              float x0, x1, x2, x3;
              tc_fma2(x0, x1, s[e], s[e + 1], c, n.x, n.y);
              tc_fma2(x2, x3, s[e + 2], s[e + 3], c, n.z, n.w);
              tc_add2(sum[0], sum[1], exp2_approx(x0), exp2_approx(x1));
              tc_add2(sum[2], sum[3], exp2_approx(x2), exp2_approx(x3));
            }
          }
        } else {
          const int lo = key.see0 - r0, hi = min(key.see1 - r0, R);  // this key's columns
          const int q1 = min(any1 - r0, R);
#pragma unroll 1
          for (int q = max(any0 - r0, 0) & ~31; q < q1; q += 32) {
            const uint32_t four = (q & 64) ? ((q & 32) ? adds.w : adds.z) : ((q & 32) ? adds.y : adds.x);
            const uint32_t see = four & low_bits(hi - q) & ~low_bits(lo - q);
            uint32_t v[2][16];
            tc_ld16_start(at + q, v[0]);
            tc_ld16_start(at + q + 16, v[1]);
            tc_ld16_wait(v[0]);
            tc_ld16_wait(v[1]);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              uint32_t (&s)[16] = v[e / 16];
              const float4 n = neg[q / 4 + e / 4];
              float x[4];
              tc_fma2(x[0], x[1], s[e % 16], s[e % 16 + 1], c, n.x, n.y);
              tc_fma2(x[2], x[3], s[e % 16 + 2], s[e % 16 + 3], c, n.z, n.w);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float y = exp2_approx(x[i]);
                if ((see >> (e + i)) & 1u) sum[i] += y;
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(bar(sh.s_empty[place]));
        place = place == 0 ? 2 : place - 1;  // two places on
        if (place != 2) ++turn;
      }
      const bool draws = key.page >= 0 && key.page < a.num_pages;
      lost = lost || !draws;
      if (key.w && !cta_abort.raised()) 
        *key.w = key.old + (draws ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.0f);
    };
    // (two by turns: a copy of one whose loads are on their way would wait for them)
    Walk walk;
    Key x, y;
    bool more = first_item(walk);
    if (more) x = key_of(walk.it);
    while (more && !given_up()) {
      more = next_item(walk);
      if (more) y = key_of(walk.it);
      item_sum(x);
      if (!more || given_up()) break;
      more = next_item(walk);
      if (more) x = key_of(walk.it);
      item_sum(y);
    }
    if (lost && a.status) atomicOr(a.status, kStatusBadSlot);
  } else if (warp < 16) {
    // -------------------------------------------------------------- keys
    const int r = tid - 256;
    const int page_blocks = a.page_size / 16;
    const long long page_bytes = static_cast<long long>(a.num_kv_heads) * page_blocks * B::kBytes;
    // A walk two items ahead asks for the page of this thread's key, one ahead for its codes.
    struct Codes {
      bool used;
      uint4 codes[D / 32];
      uint32_t scales[D / 64];
    };
    Walk walk;
    bool more = first_item(walk);
    int page, in_page = 0;
    bool exists, used = false;  // of the item looked up last
    auto look_up = [&]() {
      exists = more;
      page = -1;
      if (!more) return;
      const TcItem& it = walk.it;
      used = it.rows > 0;
      const int j = it.kt * kTcKeys + r;
      if (j < it.seq.end && j >= it.seq.first_key(0, a.window)) {
        const int pg = page_of(j), in = j - pg * a.page_size;
        page = __ldg(a.page_table + it.b * a.table_stride + pg);
        in_page = (it.h * page_blocks + in / 16) * B::kBytes;
      }
      more = next_item(walk);
    };
    auto fetch = [&](Codes& x) -> bool {  // of the item looked up last; then the next is
      x.used = used;
      const bool there = exists;
      const uint8_t* blk = page >= 0 && page < a.num_pages ? a.cache + page * page_bytes + in_page : nullptr;
#pragma unroll
      for (int c = 0; c < D / 32; ++c)  // (an item's keys begin at a multiple of 16)
        x.codes[c] = blk ? __ldg(reinterpret_cast<const uint4*>(blk + (r & 15) * B::kCodeRow) + c)
                         : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        x.scales[c] = blk ? __ldg(reinterpret_cast<const uint32_t*>(blk + B::kKScale + (r & 15) * B::kScaleRow) + c)
                          : 0u;
      look_up();
      return there;
    };
    uint32_t n = 0;  // items with products so far
    const uint32_t tK = taddr + (static_cast<uint32_t>((warp & 3) * 32) << 16) + ((warp - 8) >> 2) * (D / 2);
    auto widen = [&](const Codes& x) {
      if (!x.used) return;
      bool ok = true;
      if (n >= 1) ok = cta_abort.wait(bar(sh.k_empty), (n - 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {  // 32 dimensions: two scales, 16 columns
        const uint32_t h = e4m3x2_to_f16(x.scales[c / 2] >> (16 * (c & 1)));
        const uint32_t f[2] = {__byte_perm(h, h, 0x1010), __byte_perm(h, h, 0x3232)};
        const uint32_t y[4] = {x.codes[c].x, x.codes[c].y, x.codes[c].z, x.codes[c].w};
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t u[4];
          e2m1x8_to_f16(y[e], u);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u[i] = hmul2(u[i], f[e / 2]);
            if constexpr (!F16) {
              const float2 w = unpack_f16x2(u[i]);
              u[i] = pack_bf16x2(w.x, w.y);
            }
            v[4 * e + i] = u[i];
          }
        }
        tc_st16(tK + 16 * c, v);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(bar(sh.k_full));
      ++n;
    };
    Codes x[2];
    look_up();
    bool here = fetch(x[0]);
    while (here && !given_up()) {
      const bool then = fetch(x[1]);
      widen(x[0]);
      if (!then || given_up()) break;
      here = fetch(x[0]);
      widen(x[1]);
    }
  } else if (warp > 16) {
    // -------------------------------------------------------------- rows
    constexpr int CHUNKS = D / 8, AT_ONCE = 32 / CHUNKS;  // 16-byte chunks of a row, rows of a warp's copy
    const int r = tid - 17 * 32, ch = lane % CHUNKS;
    const uint32_t magic = ((1u << 20) + group - 1) / group;  // n / group = n * magic >> 20 for n < 2^9
    bool odd_path = false;
    uint32_t t = 0;
    Walk walk;
    for (bool more = first_item(walk); more && !given_up(); more = next_item(walk)) {
      const TcItem& it = walk.it;
      const uint16_t* q_head = a.q + static_cast<long long>(it.h) * group * D + 8 * ch;
      for (int r0 = it.row0; r0 < it.row0 + it.rows; r0 += R, ++t) {
        const int st = t % kTcStages, slot = t % kTcAhead;
        const int cols = min(it.row0 + it.rows - r0, R);
        const int i0 = r0 / group, g0 = r0 - i0 * group;  // the tile's first row and head
        // the place of the tile's packed row c in q (below 0: none) and its head
        auto place = [&](int c, int& head) {
          const int i = static_cast<int>((static_cast<uint32_t>(g0 + c) * magic) >> 20);
          head = g0 + c - i * group;
          return it.seq.row_in_q(a, it.b, i0 + i);
        };
        float lse[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int c = r + u * kTcCopiers;
          lse[u] = -INFINITY;
          if (c < cols) {
            int head;
            const int at = place(c, head);
            if (at >= 0) lse[u] = __ldg(a.lse + static_cast<long long>(at) * a.num_q_heads + it.h * group + head);
            else odd_path = true;
          }
        }
        if (t >= kTcStages) cta_abort.wait(bar(sh.q_empty[st]), (t / kTcStages - 1) & 1);
        __syncwarp();
        const uint32_t to = sbase + st * kTile;
        const bool stop = given_up();
        if (p.by_tma) {
          if (warp == 17 && !stop && tc_elect()) {
            mbar_arrive_expect_tx(bar(sh.q_full[st]), static_cast<uint32_t>(ATOMS * R * 128));
#pragma unroll
            for (int x = 0; x < ATOMS; ++x)
              tma_load_3d(to + x * kAtom, &params.q, 64 * x, it.h * group, it.seq.q0 + i0, bar(sh.q_full[st]));
          }
          __syncwarp();
        } else {
          const int padded = (cols + 15) & ~15;
#pragma unroll 4
          for (int c = (warp - 17) * AT_ONCE + lane / CHUNKS; c < padded; c += 3 * AT_ONCE) {
            int head;
            const int at = place(min(c, cols - 1), head);
            const bool real = c < cols && at >= 0;
            cp_async_16(to + (ch >> 3) * kAtom + swz128(c, ch & 7), q_head + (real ? at : 0) * a.q_stride + head * D,
                        real);
          }
          // (the copies arrive themselves as they land; the products' warp fences)
          if (!stop) cp_async_mbar_arrive(bar(sh.q_full[st]));
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int c = r + u * kTcCopiers;
          if (c < kTcRows) {  // (a whole warp, or none of it)
            sh.neg[slot][c] = lse[u] == -INFINITY ? -INFINITY : -(lse[u] * kTcLog2e);
            const uint32_t adds = __ballot_sync(0xffffffffu, c >= cols || lse[u] != -INFINITY);
            if (lane == 0) sh.adds[slot][c / 32] = adds;
          }
        }
        __syncwarp();
        if (lane == 0 && !stop) mbar_arrive(bar(sh.l_full[slot]));
      }
    }
    // (a call that gives up waits for the boxes that it has asked for)
    if (p.by_tma && warp == 17 && lane == 0 && cta_abort.raised())
      for (uint32_t x = t > kTcStages ? t - kTcStages : 0; x < t; ++x)
        mbar_drain(bar(sh.q_full[x % kTcStages]), (x / kTcStages) & 1, p.wait_limit_ns);
    __syncwarp();
    if (odd_path && a.status) atomicOr(a.status, kStatusBadLength);
  } else {
    // -------------------------------------------------------------- products
    uint32_t t = 0, n = 0, place = 0, turn = 0;
    Walk walk;
    bool ok = true;
    for (bool more = first_item(walk); ok && more; more = next_item(walk)) {
      const TcItem& it = walk.it;
      if (it.rows == 0) continue;
      ok = __all_sync(0xffffffffu, cta_abort.wait(bar(sh.k_full), n & 1));
      for (int left = it.rows; ok && left > 0; left -= R, ++t) {
        const int st = t % kTcStages;
        ok = __all_sync(0xffffffffu, cta_abort.wait(bar(sh.q_full[st]), (t / kTcStages) & 1));
        if (!ok) break;
        fence_proxy_async();  // (rows that copies of other threads wrote)
        // (of a full tile, all columns are summed, those behind its last row too: products of zeros)
        const int columns = left >= R ? kTcRows : (left + 15) & ~15;
        const uint32_t idesc = kIdesc | (static_cast<uint32_t>(columns >> 3) << 17);
        const uint64_t dq = umma_desc_sw128(sbase + st * kTile, 16, 1024);
#pragma unroll
        for (int s = 0; s < 2; ++s) {  // (one key tile's sums run under the other's products)
          if (turn > 0) ok = __all_sync(0xffffffffu, cta_abort.wait(bar(sh.s_empty[place]), (turn - 1) & 1));
          if (!ok) break;
          tc_fence_after();
          if (tc_elect()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * kAtom + (kk & 3) * 32) >> 4;
              tc_mma_ts(taddr + kColS + place * kTcRows, taddr + s * (D / 2) + 8 * kk, dq + off, idesc, kk != 0 ? 1u : 0u);
            }
            umma_commit(bar(sh.s_full[place]));
            if (s == 1) {
              umma_commit(bar(sh.q_empty[st]));
              if (left <= R) umma_commit(bar(sh.k_empty));
            }
          }
          __syncwarp();
          if (++place == kTcPlaces) place = 0, ++turn;
        }
      }
      ++n;
    }
    if (cta_abort.raised()) {  // the products still running end before the TMEM goes
      if (tc_elect()) {
        umma_commit(bar(sh.drain));
        mbar_drain(bar(sh.drain), 0, p.wait_limit_ns);
      }
      __syncwarp();
    }
  }
  asm volatile("cp.async.wait_all;\n" ::: "memory");  // (a call that gave up may have some on their way)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(512u)
                 : "memory");
  if (tid == 0 && cta_abort.raised() && a.status) atomicOr(a.status, kStatusTimeout);
}

namespace {
template <bool PATH>
const void* tc_kernel(int head_dim, bool f16) {
  if (head_dim == 64)
    return f16 ? reinterpret_cast<const void*>(lora_kv4_weights_tc_kernel<64, true, PATH>)
               : reinterpret_cast<const void*>(lora_kv4_weights_tc_kernel<64, false, PATH>);
  return f16 ? reinterpret_cast<const void*>(lora_kv4_weights_tc_kernel<128, true, PATH>)
             : reinterpret_cast<const void*>(lora_kv4_weights_tc_kernel<128, false, PATH>);
}
}  // namespace

int launch_kv4_weights_tc(const Kv4WeightsArgs& a, int max_packed_rows, bool f16, cudaStream_t stream) {
  const void* fn = a.path ? tc_kernel<true>(a.head_dim, f16) : tc_kernel<false>(a.head_dim, f16);
  const size_t smem = 1024 + kTcStages * static_cast<size_t>(a.head_dim / 64) * 128 * 128 + sizeof(TcShared);
  if (ensure_smem_attr(fn, smem) != 0) return -6;
  const int sms = std::min(device_sm_count(), kTcCtasMax);
  if (sms <= 0) return -6;
  TcParamsTma p;
  p.p.a = a;
  p.p.max_packed_rows = max_packed_rows;
  const int group = a.num_q_heads / a.num_kv_heads;
  p.p.tile_rows = group <= kTcRows ? kTcRows / group * group : kTcRows;
  p.p.by_tma = !a.path && group <= kTcRows &&
               make_tmap_3d(&p.q, a.q, a.head_dim, a.num_q_heads, a.max_num_tokens, a.head_dim * 2ll,
                            a.q_stride * 2, group, kTcRows / group) == 0;
  const unsigned long long page_blocks = a.page_size / 16;
  p.p.page_magic = ((1ull << 36) + page_blocks - 1) / page_blocks;
  p.p.wait_fault = wait_fault() ? 1 : 0;
  p.p.wait_limit_ns = p.p.wait_fault ? kTestWaitLimitNs : kWaitLimitNs;
  return launch_pdl(fn, dim3(sms), dim3(kTcThreads), smem, stream, 0, &p);
}

}  // namespace grg
