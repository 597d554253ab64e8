// Attention over the 4-bit paged cache for sequences with many query rows
// (chunks of prefill), on the 5th-generation tensor cores.
//
// An item is 256 packed rows (row x head of one key head) of a sequence, as two
// tiles of 128, against tiles of 128 keys:
//   S_t = Q_t K^T (M = 128 rows, N = 128 keys), p = 2^(S c - m), O_t += P_t V
// with S_t and O_t in TMEM (2 x 128 + 2 x D columns) and P_t written over S_t as
// fp16, from where the second product reads it.  The codes times their e4m3
// scales are exact in fp16, so only P is rounded.
//
// Warp roles (12 warps of 168 registers, one CTA per SM, persistent):
//  - warps 0-3 and 4-7, softmax of tile 0 and 1: a thread owns a row.  Per key tile
//    it reads S, forms p in one pass against a running reference m (moved, and O
//    rescaled, only when a tile's sum shows that p may leave fp16's range) and stores
//    P; then one lane of the tile's first warp issues O += P V and the next S, so
//    that one tile's products run under the other tile's softmax.  At an item's end the
//    next item's queries are copied to shared memory while the rows of O go out; then
//    they are turned into fp16 (bf16: scaled by a power of two per row) in place.
//  - warps 8-11, keys and values: a thread owns a key of the tile.  It loads
//    the key's codes and scales into registers a tile ahead (the page's number two
//    ahead), and writes the fp16 values into the swizzled operand tiles (two stages
//    each for K and V).
// Work: the key tiles of all items in one line, cut into equal runs, one per CTA;
// an item that was cut leaves (m, l, O) partials, joined in run order by the last
// of its CTAs to finish (as in kv4_decode.cuh).  Short items stay whole.
//
// Measured (GB300, bf16): 6 chunks of 700 to 2000 rows over 2000 to 5000 keys, 32 / 8
// heads of 128: 314 us, 1095 TFLOP/s (0.57 of measured), fp16 304 us; heads of 64 264 and
// 257 us; one prompt of 8192 tokens, 32 / 32 heads of 128: 462 us, 1190 TFLOP/s.  Bound by
// the chain softmax (1400 cycles a tile of
// 128 x 128), barrier and issue, two products (1024 at the tensor core's rate): 3390
// cycles a key tile of two row tiles, whose products alone take 2048.  The issuing warp
// is held until its products are nearly done, so its own softmax starts some 400 cycles
// late; a warp for the issue alone would leave 128 registers a thread, and two threads a
// row (96 registers) took 361 us.  An item's start and end cost about five key tiles.
//
// TREE (rows that see what their masks name) differs where tiles are masked: a thread's row
// takes 32 keys' bits from its mask.  32 trees of 64 rows over up to 4000 keys, 32 / 8 heads of 128: 100
// us; 2 of 60 over up to 100000, 32 / 32 heads: 387 us.  Trees pack to one or two row tiles, so that
// the warps that widen keys (2600 to 3000 cycles a tile of 128) are what most wait for, not the products.
#pragma once

#include "kv4_attention.cuh"
#include "kv4_attention.h"
#include "launch.h"

namespace grg {

namespace {
constexpr int kPreThreads = 12 * 32;  // (168 registers each)
constexpr int kPreWarps = kPreThreads / 32;
constexpr int kPreCtasMax = 160;  // CTAs that the workspace has room for
constexpr int kPreRows = 256;     // packed rows of an item
constexpr int kPreKeys = 128;     // keys of a tile
// What the line counts: a key tile of two row tiles, of one, and an item's start and
// end (12: 4000 rows in a window of 1000 123.8 us, 16: 118.4 us; 8 and 28 cost 3 % on 6
// chunks).
constexpr int kCostTwo = 3, kCostOne = 2, kCostItem = 16;
constexpr int kWholeTiles = 8;    // an item of so few key tiles is not cut for the sake of idle CTAs
constexpr int kStagePitch = 80;   // bytes of a staged row: 32 values of 16 bits, and 16 against bank conflicts
constexpr float kPreLog2e = 1.4426950408889634f;
constexpr float kPreLn2 = 0.6931471805599453f;
constexpr float kPreNoKey = -3e38f;     // the running reference before any key
constexpr float kPreFar = 16777216.0f;  // 2^24: from here on a reference's own rounding is half a unit or more
constexpr float kPreTaken = 1e-30f;     // stands for a reference that has been taken off S: as good as 0

struct PrefillParams {
  Kv4AttnArgs a;
  uint32_t* counters;   // [kPreCtasMax], zero between calls
  float4* part_o;       // [2 * kPreCtasMax][2 tiles][D / 4][128 rows]
  float2* part_ml;      // [2 * kPreCtasMax][256]
  int max_packed_rows;  // sequences with no more packed rows are not this kernel's
  unsigned long long wait_limit_ns;
  int wait_fault;
};

// An item's keys [lo, hi), hi = 0 where no row sees a key, and its key tiles [kt0, kt0 + nt).
struct PreItem {
  int lo, hi, nt;
  int cost;  // of a key tile
  __device__ __forceinline__ int kt0() const { return lo / kPreKeys; }
  __device__ __forceinline__ int size() const { return kCostItem + nt * cost; }
};
template <bool TREE>
__device__ __forceinline__ PreItem pre_item(const Kv4Seq& s, int group, int rt, int window) {
  // (packed rows fit 32 bits: 2^22 tokens of 2^8 heads)
  const uint32_t first = static_cast<uint32_t>(rt) * kPreRows;
  const uint32_t rows = min(static_cast<uint32_t>(s.take * group) - first, static_cast<uint32_t>(kPreRows));
  const int i0 = static_cast<int>(first / static_cast<uint32_t>(group));
  const int i1 = static_cast<int>((first + rows - 1) / static_cast<uint32_t>(group));
  const int hi = s.keys_end<TREE>(i1), lo = s.keys_first<TREE>(i0, window);
  PreItem it;
  it.lo = lo;
  it.hi = hi > lo ? hi : 0;
  it.nt = hi > lo ? (hi - 1) / kPreKeys - it.kt0() + 1 : 1;  // (hi may be 2^31 - 16)
  it.cost = rows > 128 ? kCostTwo : kCostOne;
  return it;
}
// What a CTA does of an item.
struct PrePart {
  Kv4Seq seq;
  PreItem item;
  int b, h, rt;
  int o, take;   // key tiles [o, o + take) of the item
  long long at;  // the item's place in the line
};

// Shared memory behind the operand tiles.
struct PreShared {
  uint64_t s_full[2];     // a tile's scores are there
  uint64_t o_done[2][2];  // [tile][stage]: its second product on that stage is done
  uint64_t k_full[2], v_full[2];
  uint64_t drain[2];
  // keys of a tile that exist; four tiles deep: a tile's words are rewritten only
  // after both softmaxes have taken the tile two further on
  __align__(16) uint32_t valid[4][4];
  uint32_t taddr;
  int abort, poison, last;
  PrePart part[8][2];    // the softmax warps' parts (their registers are needed for S)
  long long u0, u_end, per;
  int whole;  // items are not cut
  __align__(16) unsigned char staged[8][32 * kStagePitch];  // of the softmax warps
  long long prefix[2][kPreThreads + 1];  // of the line, and of items
  long long warp_sum[2][kPreWarps];
  int most;  // key tiles of the longest item
};

__device__ __forceinline__ uint32_t pre_prmt(uint32_t a, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %1, %2;\n" : "=r"(r) : "r"(a), "r"(sel));
  return r;
}
// D[tmem] (+)= A[tmem] * B[shared].
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 32 consecutive 32-bit columns of this thread's TMEM lane: the load, and the
// wait for every load so far (the registers hold nothing before it).
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}
// (a0, a1) * (b, b) + (c, c) and (a0, a1) + (b0, b1), two fp32 at a time.
__device__ __forceinline__ void fma2(float& x, float& y, uint32_t a0, uint32_t a1, float b, float c) {
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 c, {%5, %5};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(x), "=f"(y)
      : "r"(a0), "r"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n add.rn.f32x2 a, a, b;\n"
      " mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}
// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// The same, and whether any of the threads says so.
__device__ __forceinline__ bool pre_barrier_any(int id, int threads, bool says) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(says ? 1u : 0u), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void pre_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

}  // namespace

template <int D, bool F16, bool TREE>
__global__ void __launch_bounds__(kPreThreads, 1)
    lora_kv4_prefill_kernel(const __grid_constant__ PrefillParams p) {
  using B = Kv4Block<D>;
  constexpr int ATOMS = D / 64;                      // 128-byte atoms of a row
  constexpr uint32_t kTile = ATOMS * 128 * 128;      // bytes of an operand tile of 128 rows
  constexpr uint32_t kAtom = 128 * 128;
  constexpr uint32_t kOffK = 2 * kTile, kOffV = 4 * kTile, kOffShared = 6 * kTile;
  // D fp32, A and B fp16; M = 128; the second product's B is MN-major
  constexpr uint32_t kIdescS = (1u << 4) | (static_cast<uint32_t>(kPreKeys >> 3) << 17) | (8u << 24);
  constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) | (8u << 24);
  constexpr uint32_t kColS = 0, kColO = 2 * kPreKeys;  // TMEM columns of S (and P) and O
  constexpr uint32_t kCols = 512;

  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (sbase - raw);
  PreShared& sh = *reinterpret_cast<PreShared*>(smem + kOffShared);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform, and known to be
  const Kv4AttnArgs& a = p.a;
  const int group = a.num_q_heads / a.num_kv_heads;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.o_done[0][i]), 1);
      mbar_init(smem_u32(&sh.o_done[1][i]), 1);
      mbar_init(smem_u32(&sh.k_full[i]), 4 + (p.wait_fault ? 1 : 0));
      mbar_init(smem_u32(&sh.v_full[i]), 4);
    }
    mbar_init(smem_u32(&sh.drain[0]), 1);
    mbar_init(smem_u32(&sh.drain[1]), 1);
    fence_mbar_init();
    sh.abort = 0;
    sh.poison = 0;
    sh.most = 0;
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     smem_u32(&sh.taddr)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  const CtaAbort cta_abort{&sh.abort, p.wait_limit_ns};
  pdl_wait();
  pdl_launch_dependents();

  // ---- the line of units (key tiles): a prefix sum over the threads' runs of
  // sequences; where there are few, a group of lanes shares a sequence's row tiles,
  // and its first lane has the sum (one prompt of 8192 rows: 13 thousand cycles
  // with a thread a sequence)
  const int per_thread = (a.num_seqs + kPreThreads - 1) / kPreThreads;
  int group_lanes = 1;
  while (group_lanes < 32 && 2 * group_lanes * a.num_seqs <= kPreThreads) group_lanes *= 2;
  auto mine_of = [&](const Kv4Seq& s) {
    return !s.few<TREE>(a, group, p.max_packed_rows);
  };
  auto tiles_of = [&](const Kv4Seq& s) {
    return (s.take * group + kPreRows - 1) / kPreRows;
  };
  // units of one key head, the row tiles from `from` on in steps of `step`
  auto head_units = [&](const Kv4Seq& s, int from, int step, int& most) -> long long {
    long long n = 0;
    if (mine_of(s)) {
      const int nr = tiles_of(s);
      for (int rt = from; rt < nr; rt += step) {
        const PreItem it = pre_item<TREE>(s, group, rt, a.window);
        n += it.size();
        most = max(most, it.nt);
      }
    }
    return n;
  };
  long long mine[2] = {0, 0};
  int most = 0;
  {
    const int sub = lane & (group_lanes - 1);
    for (int i = 0; i < per_thread; ++i) {
      const int b = tid / group_lanes * per_thread + i;
      if (b < a.num_seqs) {
        const Kv4Seq s = Kv4Seq::of(a, b);
        mine[0] += head_units(s, sub, group_lanes, most) * a.num_kv_heads;
        if (sub == 0 && mine_of(s)) mine[1] += static_cast<long long>(tiles_of(s)) * a.num_kv_heads;
      }
    }
    for (int o = 1; o < group_lanes; o <<= 1) mine[0] += __shfl_xor_sync(0xffffffffu, mine[0], o);
    if (sub != 0) mine[0] = 0;
  }
  long long run[2] = {mine[0], mine[1]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const long long v = __shfl_up_sync(0xffffffffu, run[i], o);
      if (lane >= o) run[i] += v;
    }
  if (lane == 31) sh.warp_sum[0][warp] = run[0], sh.warp_sum[1][warp] = run[1];
  most = __reduce_max_sync(0xffffffffu, most);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (lane == 0 && most > 0) atomicMax(&sh.most, most);
  long long all[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    long long before = 0;
#pragma unroll
    for (int w = 0; w < kPreWarps; ++w) {
      if (w < warp) before += sh.warp_sum[i][w];
      all[i] += sh.warp_sum[i][w];
    }
    sh.prefix[i][tid] = before + run[i] - mine[i];
    if (tid == 0) sh.prefix[i][kPreThreads] = all[i];
  }
  __syncthreads();
  const uint32_t taddr = sh.taddr;

  if (tid == 0) {
    // Short items stay whole where there is a CTA for each: cutting one costs its
    // join, about as long as kWholeTiles tiles.  Else the line is cut into equal
    // runs (no shorter than a tile, so every run inside an item has one of its tiles).
    sh.whole = sh.most <= kWholeTiles && all[1] <= gridDim.x;
    sh.per = sh.whole ? 1 : max(quotient(all[0] + gridDim.x - 1, gridDim.x),
                                static_cast<long long>(kCostTwo));
    sh.u0 = blockIdx.x * sh.per;
    sh.u_end = min(sh.u0 + sh.per, sh.whole ? all[1] : all[0]);
  }
  __syncthreads();

  // A tile is the run's in which its place begins.
  auto set_part = [&](PrePart& q) {
    q.item = pre_item<TREE>(q.seq, group, q.rt, a.window);
    auto tiles_before = [&](long long x) {  // tiles that begin before place x
      const long long far = x - q.at - kCostItem;
      if (far <= 0) return 0;
      const uint32_t n = far > (1 << 30) ? 1u << 30 : static_cast<uint32_t>(far);
      const uint32_t k = q.item.cost == kCostTwo ? (n + kCostTwo - 1) / kCostTwo : (n + kCostOne - 1) / kCostOne;
      return min(static_cast<int>(k), q.item.nt);
    };
    q.o = sh.whole ? 0 : tiles_before(sh.u0);
    q.take = sh.whole ? q.item.nt : tiles_before(sh.u_end) - q.o;
  };
  auto next_part = [&](PrePart& q) -> bool {
    do {
      q.at += sh.whole ? 1 : q.item.size();
      if (q.at >= sh.u_end) return false;
      if (++q.rt == tiles_of(q.seq)) {
        q.rt = 0;
        if (++q.h == a.num_kv_heads) {
          q.h = 0;
          do q.seq = Kv4Seq::of(a, ++q.b);
          while (!mine_of(q.seq));
        }
      }
      set_part(q);
    } while (q.take == 0);
    return true;
  };
  auto first_part = [&](PrePart& q) -> bool {
    const long long u0 = sh.u0;
    if (u0 >= sh.u_end) return false;
    const long long* prefix = sh.prefix[sh.whole ? 1 : 0];
    const int lo = last_not_past<kPreWarps>(prefix, u0, lane);
    int ignored = 0;
    long long off = u0 - prefix[lo], n;
    q.b = lo / group_lanes * per_thread;
    while (true) {
      q.seq = Kv4Seq::of(a, q.b);
      if (sh.whole) {
        n = mine_of(q.seq) ? tiles_of(q.seq) : 0;
      } else {  // by all lanes
        n = head_units(q.seq, lane, 32, ignored);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      }
      if (off < n * a.num_kv_heads) break;
      off -= n * a.num_kv_heads;
      ++q.b;
    }
    q.h = static_cast<int>(quotient(off, n));
    off -= q.h * n;
    q.rt = 0;
    if (sh.whole) {
      q.rt = static_cast<int>(off);
      off = 0;
    } else {  // 32 row tiles at a time
      const int nr = tiles_of(q.seq);
      while (true) {
        const int size = q.rt + lane < nr ? pre_item<TREE>(q.seq, group, q.rt + lane, a.window).size() : 0;
        int to = size;  // sizes up to this lane's
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, to, o);
          if (lane >= o) to += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, off < to);
        const int at = past ? __ffs(past) - 1 : 31;
        off -= __shfl_sync(0xffffffffu, past ? to - size : to, at);
        q.rt += past ? at : 32;
        if (past) break;
      }
    }
    q.at = u0 - off;
    set_part(q);
    return q.take > 0 || next_part(q);
  };
  auto live_rows = [&](const PrePart& q) {
    return min(q.seq.take * group - q.rt * kPreRows, kPreRows);
  };
  auto bar = [&](uint64_t& b) { return smem_u32(&b); };

  PrePart q;
  if (first_part(q)) {
    if (warp < 8) {
      // -------------------------------------------------------------- softmax
      const int t = warp >> 2;                    // tile
      const int row_in_tile = (warp & 3) * 32 + lane;  // and TMEM lane
      const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t tS = taddr + lane_base + kColS + t * kPreKeys;
      const uint32_t tO = taddr + lane_base + kColO + t * D;
      const uint32_t sS = taddr + kColS + t * kPreKeys, sO = taddr + kColO + t * D;
      uint32_t ns = 0;          // first products of this tile so far
      uint32_t no[2] = {0, 0};  // and second ones, by stage
      uint32_t it = 0;          // key tiles so far (the stages of K and V)
      // The products, issued by one lane of the tile's first warp, in the order
      // S(0), O(0), S(1), O(1), ...: the tensor core takes one tile's in turn, so S
      // never overwrites a P still to be read.  A key tile's stages of K and V are free
      // when the second products of both tiles (all that are active) are done: until
      // then its scores can be formed once more.
      auto scores = [&](uint32_t st) {  // on stage st
        const uint64_t dq = umma_desc_sw128(sbase + t * kTile, 16, 1024);
        const uint64_t dk = umma_desc_sw128(sbase + kOffK + st * kTile, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {  // (addresses count in 16 bytes)
          const uint32_t off = ((kk >> 2) * kAtom + (kk & 3) * 32) >> 4;
          umma_f16(sS, dq + off, dk + off, kIdescS, kk != 0 ? 1u : 0u);
        }
        umma_commit(bar(sh.s_full[t]));
      };
      auto values = [&](uint32_t st, bool add) {
        const uint64_t dv = umma_desc_sw128(sbase + kOffV + st * kTile, kAtom, 1024);
        umma_f16_ts(sO, sS, dv, kIdescO, add ? 1u : 0u);
#pragma unroll
        for (int kk = 1; kk < kPreKeys / 16; ++kk)
          umma_f16_ts(sO, sS + 8 * kk, dv + ((kk * 16 * 128) >> 4), kIdescO, 1u);
        umma_commit(bar(sh.o_done[t][st]));
      };
      auto have_k = [&](uint32_t i) {
        return __all_sync(0xffffffffu, cta_abort.wait(bar(sh.k_full[i & 1]), (i >> 1) & 1));
      };
      auto have_v = [&](uint32_t i) {
        return __all_sync(0xffffffffu, cta_abort.wait(bar(sh.v_full[i & 1]), (i >> 1) & 1));
      };
      // waits for the second product on stage st that was issued last
      auto settled = [&](uint32_t st) {
        cta_abort.wait(bar(sh.o_done[t][st]), ((st ? no[1] : no[0]) - 1) & 1);
        __syncwarp();
        tc_fence_after();
      };
      // This thread's row of a part.
      struct Row {
        int nact;     // tiles of the part that have rows
        int pos, lo;  // its position, and the first key that it sees
        float cf;     // what turns its products into scores in units of log2
        int tok;      // (TREE) the row in q
      };
      // Where it lies in q and out (rows past the end repeat the last).
      struct Place {
        int i, tok, head;
        bool live;
      };
      auto place = [&](const PrePart& w) {
        Place x;
        const int live = live_rows(w), r = t * 128 + row_in_tile;
        x.live = r < live;
        const int pr = w.rt * kPreRows + min(r, live - 1);
        x.i = pr / group;
        x.head = w.h * group + pr - x.i * group;
        x.tok = w.seq.q0 + x.i;
        return x;
      };
      // Starts a part in two steps.  First its rows of q are copied to shared memory:
      // asynchronously, while the rows of the part before go out.
      // The warp's 32 rows, D / 8 lanes a row and 256 / D rows at a time, so that a row's
      // reads are neighbours.
      constexpr int LANES = D / 8, AT_ONCE = 32 / LANES, PASSES = 32 / AT_ONCE;
      auto chunk = [&](int i2) {  // the 16 bytes of q that this thread copies in a pass
        const int r = i2 * AT_ONCE + lane / LANES, c = lane % LANES;
        return static_cast<uint32_t>(t * kTile + (c >> 3) * kAtom) + swz128((warp & 3) * 32 + r, c & 7);
      };
      auto begin_part = [&](const PrePart& w) {
        Row x;
        const Place mine_p = place(w);
        x.nact = live_rows(w) > 128 ? 2 : 1;
        x.pos = w.seq.run_last<TREE>(mine_p.i);
        x.lo = w.seq.run_first<TREE>(a, mine_p.i);
        x.tok = mine_p.tok;
        x.cf = 0.0f;
        if (t >= x.nact) return x;
#pragma unroll
        for (int i2 = 0; i2 < PASSES; ++i2) {
          const int r = i2 * AT_ONCE + lane / LANES;
          const long long tok = __shfl_sync(0xffffffffu, mine_p.tok, r);
          const int head = __shfl_sync(0xffffffffu, mine_p.head, r);
          cp_async_16(sbase + chunk(i2), a.q + tok * a.q_stride + head * D + 8 * (lane % LANES), true);
        }
        cp_async_commit();
        return x;
      };
      // Then each thread turns what it has copied into fp16, and the first product
      // starts.
      auto finish_part = [&](int nact) {
        if (t >= nact) return 0.0f;
        cp_async_wait<0>();
        float down = 1.0f;  // (fp16 rows need no factor)
        if constexpr (!F16) {
#pragma unroll 4
          for (int i2 = 0; i2 < PASSES; ++i2) {
            uint4* at = reinterpret_cast<uint4*>(smem + chunk(i2));
            const uint4 raw_q = *at;
            uint32_t z[4] = {raw_q.x, raw_q.y, raw_q.z, raw_q.w};
            // the row's largest magnitude, as 16-bit patterns (they order like the numbers)
            uint32_t top = __vmaxu2(__vmaxu2(z[0] & 0x7FFF7FFFu, z[1] & 0x7FFF7FFFu),
                                    __vmaxu2(z[2] & 0x7FFF7FFFu, z[3] & 0x7FFF7FFFu));
            top = max(top >> 16, top & 0xFFFFu);
#pragma unroll
            for (int sft = LANES / 2; sft; sft >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, sft));
            float up, dn;
            row_factor(__uint_as_float(top << 16), up, dn);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack_bf16x2(z[e]);
              z[e] = pack_f16x2(f.x * up, f.y * up);
            }
            dn = __shfl_sync(0xffffffffu, dn, (lane % AT_ONCE) * LANES);
            if (lane / AT_ONCE == i2) down = dn;
            *at = make_uint4(z[0], z[1], z[2], z[3]);
          }
        }
        fence_proxy_async();
        pre_barrier(2 + t, 128);
        if ((warp & 3) == 0 && have_k(it)) {
          tc_fence_after();
          const uint32_t st = __shfl_sync(0xffffffffu, it & 1, 0);
          if (elect_one()) scores(st);
        }
        __syncwarp();
        return score_factor(down, a.score_scale * kPreLog2e);
      };
      Row row = begin_part(q);
      row.cf = finish_part(row.nact);
      int slot_of_part = 0, take = q.take, first_key = (q.item.kt0() + q.o) * kPreKeys;
      if (lane == 0) sh.part[warp][0] = q;
      __syncwarp();
      while (true) {
        float m = kPreNoKey, l = 0.0f;
        // The reference before it is multiplied: one of the row's S.
        float& ref = reinterpret_cast<float*>(sh.staged[warp])[lane];
        ref = kPreNoKey;
        const bool on = t < row.nact;
        for (int j = 0; on && j < take; ++j) {
          const int key0 = first_key + j * kPreKeys;
          const int hi_j = row.pos - key0, lo_j = row.lo - key0;
          // p = 2^(s c - m) against the running reference m, in one pass over S, 32
          // keys at a time.  The tile's sum tells whether m still serves: above 2^15
          // some p may pass what fp16 holds, and the tile is done again with m moved.
          // A part's first tile looks for its maximum at once.
          // m = ref c is rounded, by up to 2^-24 of it: a factor that all of a row's p
          // share, and that cancels, but past 2^27 it alone is more than fp16 holds.  So
          // where m is far from 0 in some row of the warp (queries or a scale out of all
          // proportion) ref is taken off S first, in TMEM, which leaves 0 at the maximum
          // itself; each of the warp's tiles looks for its maximum then.  Against the
          // tile's own maximum no p is above 2, so no tile is done a third time.
          // (m == kPreTaken holds for a whole warp, with or without a vote.  With it ptxas's
          // schedule takes 319 us for 128 dimensions, 6 chunks, and 278 for 64; without it 326
          // and 262.)
          bool again = j == 0 || (D == 128 ? __any_sync(0xffffffffu, m == kPreTaken) : m == kPreTaken);
          while (true) {
            cta_abort.wait(bar(sh.s_full[t]), ns & 1);
            ++ns;
            __syncwarp();
            tc_fence_after();
            const uint4 valid = *reinterpret_cast<const uint4*>(sh.valid[(it + j) & 3]);
            const bool masked = __any_sync(0xffffffffu, hi_j < 127 || lo_j > 0 ||
                                                            (valid.x & valid.y & valid.z & valid.w) != ~0u);
            auto hide = [&](int c, uint32_t (&v)[32]) {  // keys that this row does not see
              const int h = hi_j - 32 * c, g = lo_j - 32 * c;
              uint32_t seen = c == 0 ? valid.x : c == 1 ? valid.y : c == 2 ? valid.z : valid.w;
              if constexpr (TREE) {
                seen &= tree_sees(a, sh.part[warp][slot_of_part].seq, row.tok, row.lo, key0 + 32 * c);
              } else {
                if (h < 31) seen &= h < 0 ? 0u : (2u << h) - 1u;
                if (g > 0) seen &= g > 31 ? 0u : ~0u << g;
              }
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((seen >> e) & 1u)) v[e] = 0xFF800000u;  // -infinity
            };
            auto top_of = [&](float x, const uint32_t (&v)[32]) {
              float y = __uint_as_float(v[31]);
#pragma unroll
              for (int e = 0; e < 30; e += 4) {
                x = max3(x, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                if (e < 28) y = max3(y, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
              }
              return max3(x, y, __uint_as_float(v[30]));
            };
            if (__builtin_expect(again, 0)) {  // the tile's maximum first
              float mx = -INFINITY;
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                uint32_t v[32];
                tmem_ld32_start(tS + 32 * c, v);
                tmem_ld32_wait(v);
                if (masked) hide(c, v);
                mx = top_of(mx, v);
              }
              const float old = ref, to = fmaxf(old, mx);
              const float next = to == kPreNoKey ? kPreNoKey : to * row.cf;
              // (an infinity of S is a row whose q is not finite: NaN either way)
              const bool far = __any_sync(0xffffffffu, fabsf(next) >= kPreFar && fabsf(to) < -kPreNoKey);
              if (__any_sync(0xffffffffu, to > old && old != kPreNoKey)) {
                // O takes the new reference
                settled((it + j + 1) & 1);
                const float f = exp2_approx(far || m == kPreTaken ? (old - to) * row.cf : m - next);
                l *= f;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                  uint32_t r[32];
                  tmem_ld32_start(tO + 32 * c, r);
                  tmem_ld32_wait(r);
#pragma unroll
                  for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                  tmem_st16(tO + 32 * c, r);
                  tmem_st16(tO + 32 * c + 16, r + 16);
                }
              }
              ref = to;
              m = far ? kPreTaken : next;
              if (far) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                  uint32_t v[32];
                  tmem_ld32_start(tS + 32 * c, v);
                  tmem_ld32_wait(v);
#pragma unroll
                  for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) - to);
                  tmem_st16(tS + 32 * c, v);
                  tmem_st16(tS + 32 * c + 16, v + 16);
                }
                tmem_wait_st();
              }
            }
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            uint32_t v[2][32];
            tmem_ld32_start(tS, v[0]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t (&x)[32] = v[c & 1];
              tmem_ld32_wait(x);
              if (c < 3) tmem_ld32_start(tS + 32 * (c + 1), v[(c + 1) & 1]);
              if (__builtin_expect(masked, 0)) hide(c, x);
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float y, z;
                fma2(y, z, x[e], x[e + 1], row.cf, -m);
                y = exp2_approx(y), z = exp2_approx(z);
                add2(sum[e & 2], sum[(e & 2) + 1], y, z);
                w[e / 2] = pack_f16x2(y, z);
              }
              tmem_st16(tS + 16 * c, w);
            }
            const float tile_sum = (sum[0] + sum[1]) + (sum[2] + sum[3]);
            // what the products need is waited for while the other warps finish
            bool ready = true;
            if ((warp & 3) == 0) {
              const uint32_t i = it + j;
              const bool v_there = mbar_try_wait(bar(sh.v_full[i & 1]), (i >> 1) & 1);
              const bool k_there = j + 1 == take || mbar_try_wait(bar(sh.k_full[(i + 1) & 1]), ((i + 1) >> 1) & 1);
              ready = v_there && k_there && !cta_abort.raised();
              if (!__all_sync(0xffffffffu, ready)) ready = have_v(i) && (j + 1 == take || have_k(i + 1));
            }
            tmem_wait_st();
            tc_fence_before();
            // the tile's P is there, or some row wants it again
            again = pre_barrier_any(2 + t, 128, tile_sum > 32768.0f);
            if ((warp & 3) == 0 && ready) {
              tc_fence_after();
              const uint32_t st = __shfl_sync(0xffffffffu, (it + j) & 1, 0);
              const bool add = j > 0, more_keys = j + 1 < take;
              if (elect_one()) {
                if (again) {
                  scores(st);
                } else {
                  values(st, add);
                  if (more_keys) scores(st ^ 1);
                }
              }
            }
            __syncwarp();
            if (!again) {
              l += tile_sum;
              break;
            }
          }
          if ((it + j) & 1) ++no[1]; else ++no[0];
        }
        // ---- the next part starts (neither tile's warps run ahead by a part): its
        // queries are on their way while this one's rows go out
        it += take;
        const PrePart done = sh.part[warp][slot_of_part];
        const int done_lo = row.lo, done_pos = row.pos, done_nact = row.nact, done_tok = row.tok;
        if (m == kPreTaken) m = ref == kPreNoKey ? kPreNoKey : fmaxf(ref * row.cf, kPreNoKey);
        PrePart q2 = done;
        const bool more = next_part(q2);
        if (more) {
          pre_barrier(1, 256);
          row = begin_part(q2);
          slot_of_part ^= 1;
          take = q2.take, first_key = (q2.item.kt0() + q2.o) * kPreKeys;
          if (lane == 0) sh.part[warp][slot_of_part] = q2;
          __syncwarp();
        }
        if (on) {
          const Place out = place(done);
          settled((it - 1) & 1);
          uint32_t nan_blocks = 0;  // 16-dimension blocks with a NaN scale at a key of the row
          if (*reinterpret_cast<volatile int*>(&sh.poison)) {
            const int32_t* table = a.page_table + static_cast<long long>(done.b) * a.table_stride;
            // (a row of a tree sees its ancestors however far back: its run may begin behind them)
            const int k0 = max(TREE ? done.item.lo : done_lo, (done.item.kt0() + done.o) * kPreKeys);
            const int k1 = min(TREE ? done.seq.kv - 1 : done_pos,
                               (done.item.kt0() + done.o + done.take - 1) * kPreKeys + kPreKeys - 1);
            for (int key = k0; key <= k1; ++key) {
              if (TREE && !(tree_sees(a, done.seq, done_tok, done_lo, key) & 1u)) continue;
              const int page = __ldg(table + key / a.page_size), in = key % a.page_size;
              if (page < 0 || page >= a.num_pages) continue;
              const uint8_t* at = a.cache + ((static_cast<long long>(page) * a.num_kv_heads + done.h) *
                                                 (a.page_size / 16) + in / 16) * B::kBytes +
                                  B::kVScale + (in % 16) * B::kScaleRow;
              for (int e = 0; e < D / 16; ++e)
                if ((at[e] & 0x7F) == 0x7F) nan_blocks |= 1u << e;
            }
          }
          const bool all_of_it = done.take == done.item.nt;
          const int slot = static_cast<int>(blockIdx.x) * 2 + (done.o == 0 ? 1 : 0);
          unsigned char* staged = sh.staged[warp];
          // 32 dimensions of the warp's 32 rows: through shared memory, so that a
          // row's stores are neighbours (8 rows of 64 bytes at a time)
          uint16_t* dst[4];
#pragma unroll
          for (int i2 = 0; i2 < 4; ++i2) {
            const int r = 8 * i2 + (lane >> 2);
            const long long tok = __shfl_sync(0xffffffffu, out.tok, r);
            const int head = __shfl_sync(0xffffffffu, out.head, r);
            const bool store = __shfl_sync(0xffffffffu, out.live ? 1 : 0, r) && !cta_abort.raised();
            dst[i2] = store ? a.out + tok * a.out_stride + head * D + 8 * (lane & 3) : nullptr;
          }
          auto rows_out = [&](int c, const float (&v)[32], float inv) {
            unsigned char* mine_s = staged + lane * kStagePitch;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint4 w;
              w.x = pack_t<F16>(v[e] * inv, v[e + 1] * inv);
              w.y = pack_t<F16>(v[e + 2] * inv, v[e + 3] * inv);
              w.z = pack_t<F16>(v[e + 4] * inv, v[e + 5] * inv);
              w.w = pack_t<F16>(v[e + 6] * inv, v[e + 7] * inv);
              *reinterpret_cast<uint4*>(mine_s + 2 * e) = w;
            }
            __syncwarp();
#pragma unroll
            for (int i2 = 0; i2 < 4; ++i2) {
              const uint4 w = *reinterpret_cast<const uint4*>(staged + (8 * i2 + (lane >> 2)) * kStagePitch +
                                                              16 * (lane & 3));
              if (dst[i2]) *reinterpret_cast<uint4*>(dst[i2] + 32 * c) = w;
            }
            __syncwarp();
          };
          auto lse_out = [&](float top, float sum) {
            if (out.live && !cta_abort.raised() && a.lse)
              a.lse[static_cast<long long>(out.tok) * a.num_q_heads + out.head] =
                  sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kPreLn2;
          };
          // the place of 4 dimensions of this row in a slot's partials
          auto part_of = [&](long long at_slot, int c4) {
            return p.part_o + ((at_slot * 2 + t) * (D / 4) + c4) * 128 + row_in_tile;
          };
          const float inv = l == 0.0f ? 0.0f : a.v_scale / l;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float v[32];
            tmem_ld32(tO + 32 * c, v);
            if (nan_blocks) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if ((nan_blocks >> (2 * c + e / 16)) & 1u) v[e] = __uint_as_float(0x7FC00000u);
            }
            if (all_of_it) {
              rows_out(c, v, inv);
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *part_of(slot, 8 * c + e / 4) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
            }
          }
          tc_fence_before();
          if (all_of_it) {
            lse_out(m, l);
          } else {
            p.part_ml[static_cast<long long>(slot) * kPreRows + t * 128 + row_in_tile] = make_float2(m, l);
            const int threads = 128 * done_nact;
            const long long begins = done.at + kCostItem;
            const int w0 = static_cast<int>(quotient(begins, sh.per));
            const int w1 = static_cast<int>(quotient(begins + static_cast<long long>(done.item.nt - 1) * done.item.cost, sh.per));
            pre_barrier(3 + done_nact, threads);
            if (tid == 0) {
              uint32_t seen;  // releases what the barrier has gathered, acquires the others'
              asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;\n"
                           : "=r"(seen)
                           : "l"(p.counters + w0)
                           : "memory");
              sh.last = seen == static_cast<uint32_t>(w1 - w0);
              if (sh.last) p.counters[w0] = 0;
            }
            pre_barrier(3 + done_nact, threads);
            const bool last = *reinterpret_cast<volatile int*>(&sh.last) != 0;
            pre_barrier(3 + done_nact, threads);  // sh.last may change again
            if (last) {
              // every part is there: they are joined in run order
              const int runs = w1 - w0 + 1;
              auto slot_of = [&](int i) { return (static_cast<long long>(w0) + i) * 2 + (i == 0 ? 1 : 0); };
              auto ml_of = [&](int i) { return __ldcg(p.part_ml + slot_of(i) * kPreRows + t * 128 + row_in_tile); };
              float top = kPreNoKey, sum = 0.0f;
              for (int i = 0; i < runs; ++i) {
                const float2 ml = ml_of(i);
                const float to = fmaxf(top, ml.x);
                sum = sum * exp2_approx(top - to) + ml.y * exp2_approx(ml.x - to);
                top = to;
              }
              const float all_inv = sum == 0.0f ? 0.0f : a.v_scale / sum;
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                float v[32] = {};
#pragma unroll 2
                for (int i = 0; i < runs; ++i) {
                  const float f = exp2_approx(ml_of(i).x - top);
#pragma unroll
                  for (int e = 0; e < 32; e += 4) {
                    const float4 x = __ldcg(part_of(slot_of(i), 8 * c + e / 4));
                    v[e] += x.x * f, v[e + 1] += x.y * f, v[e + 2] += x.z * f, v[e + 3] += x.w * f;
                  }
                }
                rows_out(c, v, all_inv);
              }
              lse_out(top, sum);
            }
          }
        }
        if (!more) break;
        row.cf = finish_part(row.nact);
      }
      if (cta_abort.raised()) {  // the products still running end before the TMEM goes
        if ((warp & 3) == 0 && elect_one()) {  // (the thread that issued them)
          umma_commit(bar(sh.drain[t]));
          mbar_drain(bar(sh.drain[t]), 0, p.wait_limit_ns);
        }
        __syncwarp();
      }
    } else {
      // -------------------------------------------------------------- keys and values
      const int r = tid - 256;  // key of the tile
      uint4 kc[D / 32], vc[D / 32];
      uint32_t ks[D / 64], vs[D / 64];  // scale bytes
      // the walk over the key tiles: two ahead, a tile's page is asked for (and
      // nothing waits for it); one ahead, its codes and scales
      PrePart w = q;
      int wj = 0;
      bool more = true;  // the next tile to look up exists
      const uint8_t* blk = nullptr;  // this thread's key's block (null: not there)
      const int page_blocks = a.page_size / 16;
      const long long page_bytes = static_cast<long long>(a.num_kv_heads) * page_blocks * B::kBytes;
      uint32_t tiles = 0;  // two bits for this key tile, two for the next
      int page = -1, in_page = -1;  // of this thread's key in the tile looked up last; in_page -1: no such key
      auto look_up = [&](int shift) -> bool {  // tile wj of part w; then on to the next
        in_page = -1;
        if (!more) return false;
        tiles |= (live_rows(w) > 128 ? 3u : 1u) << shift;
        const int key = (w.item.kt0() + w.o + wj) * kPreKeys + r;
        if (key >= w.item.lo && key < w.item.hi) {  // (pages in front of the window may be gone)
          const int pg = key / a.page_size, in = key - pg * a.page_size;
          page = __ldg(a.page_table + static_cast<long long>(w.b) * a.table_stride + pg);
          in_page = (w.h * page_blocks + in / 16) * B::kBytes;
        }
        if (++wj == w.take) {
          wj = 0;
          more = next_part(w);
        }
        return true;
      };
      auto block = [&]() -> const uint8_t* {  // of the key looked up last
        if (in_page < 0) return nullptr;
        if (page < 0 || page >= a.num_pages) {
          if (a.status) atomicOr(a.status, kStatusBadSlot);
          return nullptr;
        }
        return a.cache + page * page_bytes + in_page;
      };
      const int key16 = r & 15;
      auto load = [&](uint4 (&codes)[D / 32], uint32_t (&scales)[D / 64], int c0, int s0) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          codes[c] = blk ? __ldg(reinterpret_cast<const uint4*>(blk + c0 + key16 * B::kCodeRow) + c)
                         : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          scales[c] = blk ? __ldg(reinterpret_cast<const uint32_t*>(blk + s0 + key16 * B::kScaleRow) + c)
                          : 0u;
      };
      auto put = [&](unsigned char* tile, const uint4 (&codes)[D / 32], const uint32_t (&scales)[D / 64]) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {  // 32 dimensions: two scales, four 16-byte chunks
          const uint32_t h = e4m3x2_to_f16(scales[c / 2] >> (16 * (c & 1)));
          const uint32_t s[2] = {pre_prmt(h, 0x1010), pre_prmt(h, 0x3232)};
          const uint32_t x[4] = {codes[c].x, codes[c].y, codes[c].z, codes[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t f[4];
            e2m1x8_to_f16(x[e], f);
            const int ch = 4 * c + e;
            *reinterpret_cast<uint4*>(tile + (ch >> 3) * kAtom + swz128(r, ch & 7)) =
                make_uint4(hmul2(f[0], s[e / 2]), hmul2(f[1], s[e / 2]),
                           hmul2(f[2], s[e / 2]), hmul2(f[3], s[e / 2]));
          }
        }
      };
      look_up(0);
      blk = block();
      load(kc, ks, B::kK, B::kKScale);
      load(vc, vs, B::kV, B::kVScale);
      bool ok = blk != nullptr;
      bool here = true, behind = look_up(2);  // this tile and the next exist
      // One lane arrives for its warp (with every thread, 319 us for 6 chunks instead of 314), and none
      // after giving up: a phase that waits for fewer arrivals than come would end the kernel.
      auto arrive = [&](uint64_t& b) {
        __syncwarp();
        if (lane == 0 && !cta_abort.raised()) mbar_arrive(bar(b));
      };
      // by stage and tile: whether the tile's product on it is to be waited for, and
      // the parity of how many there were
      uint32_t used = 0, uses = 0;
      for (uint32_t it = 0; here; ++it) {
        const int st = it & 1;
        // both tiles' products on what the stages held are done
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if ((used >> (2 * st + t)) & 1u) cta_abort.wait(bar(sh.o_done[t][st]), ((uses >> (2 * st + t)) & 1u) ^ 1u);
        __syncwarp();
        used = (used & ~(3u << (2 * st))) | ((tiles & 3u) << (2 * st));
        uses ^= (tiles & 3u) << (2 * st);
        tiles >>= 2;
        const uint32_t votes = __ballot_sync(0xffffffffu, ok);
        put(smem + kOffK + st * kTile, kc, ks);
        if (lane == 0) sh.valid[it & 3][warp - 8] = votes;
        fence_proxy_async();
        __syncwarp();
        arrive(sh.k_full[st]);
        blk = block();  // the next tile's K is on its way while V is written
        ok = blk != nullptr;
        load(kc, ks, B::kK, B::kKScale);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)  // a NaN scale must not reach rows that do not see its key
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            if (((vs[c] >> e) & 0x7Fu) == 0x7Fu) {
              sh.poison = 1;
              vs[c] &= ~(0xFFu << e);
            }
        put(smem + kOffV + st * kTile, vc, vs);
        fence_proxy_async();
        arrive(sh.v_full[st]);
        load(vc, vs, B::kV, B::kVScale);
        here = behind;
        behind = look_up(2);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(kCols)
                 : "memory");
  if (tid == 0 && cta_abort.raised() && a.status) atomicOr(a.status, kStatusTimeout);
}

namespace {
constexpr size_t kPreCounterBytes = 1024;
static_assert(kPreCtasMax * 4 <= kPreCounterBytes, "room for the counters");
}  // namespace

template <bool TREE>
int launch_kv4_prefill(const Kv4AttnArgs& a, int max_packed_rows, bool f16, cudaStream_t stream) {
  const void* fn =
      a.head_dim == 64 ? (f16 ? reinterpret_cast<const void*>(lora_kv4_prefill_kernel<64, true, TREE>)
                              : reinterpret_cast<const void*>(lora_kv4_prefill_kernel<64, false, TREE>))
                       : (f16 ? reinterpret_cast<const void*>(lora_kv4_prefill_kernel<128, true, TREE>)
                              : reinterpret_cast<const void*>(lora_kv4_prefill_kernel<128, false, TREE>));
  const size_t smem = 1024 + 6 * static_cast<size_t>(a.head_dim / 64) * 128 * 128 + sizeof(PreShared);
  if (ensure_smem_attr(fn, smem) != 0) return -6;
  const int sms = device_sm_count();
  if (sms <= 0) return -6;
  PrefillParams p;
  p.a = a;
  char* w = static_cast<char*>(a.workspace);
  p.counters = reinterpret_cast<uint32_t*>(w);
  p.part_o = reinterpret_cast<float4*>(w + kPreCounterBytes + kv4_decode_counter_bytes());
  p.part_ml = reinterpret_cast<float2*>(reinterpret_cast<char*>(p.part_o) +
                                        static_cast<size_t>(2) * kPreCtasMax * kPreRows * a.head_dim * 4);
  p.max_packed_rows = max_packed_rows;
  p.wait_fault = wait_fault() ? 1 : 0;
  p.wait_limit_ns = p.wait_fault ? kTestWaitLimitNs : kWaitLimitNs;
  return launch_pdl(fn, dim3(min(sms, kPreCtasMax)), dim3(kPreThreads), smem, stream, 0, &p);
}

}  // namespace grg
