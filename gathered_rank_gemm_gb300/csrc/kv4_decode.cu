// Attention over the 4-bit paged cache for sequences with few query rows
// (decode, drafted tokens): rows x heads of one key head are packed into groups of
// 8 * NT rows, and one pass over the group's keys forms the scores, the running
// softmax and the weighted sum of the values.
//
// Mathematics, for a block of 16 keys (mma.sync m16n8k16, fp16 operands, fp32
// accumulators; the codes times their e4m3 scales are exact in fp16):
//   S[16 keys x 8 rows] = K Q^T, the keys as M, so a group of 8 rows wastes
//   nothing;  p = 2^((S - m) c), m a running maximum of S;
//   O[16 dims x 8 rows] += V^T P, the P fragments turned by movmatrix.
// A warp holds the rows' O and the maximum and sum per row in registers; keys
// come two blocks at a time through a ring of bulk copies in shared memory, one
// copy per block (a block's codes and scales lie together).  The maximum is
// moved only when a block exceeds it by 2^6 or more: p stays below 2^6, far
// inside fp16, and the rescaling of O almost never runs.  The difference comes before
// the product: S c would be rounded by up to 2^-24 of it, which for scores past 2^27 is
// more than p's exponent has room for, while S - m is 0 at the maximum.
//
// Work: the blocks of all (sequence, row group, key head) items in one line, an
// item's fixed cost among them, cut into equal runs whatever the lengths, so one
// long sequence fills the GPU as well as many short ones.  A run goes to a
// warp, or, where an item would span many warps' runs, to a whole CTA whose warps
// share its blocks and join in shared memory; short items stay whole.  Items
// that were cut leave (m, l, O) partials in the workspace; the last of an item's
// runs to finish joins them, always in run order, so results do not depend on
// timing.
//
// Measured (GB300, bf16): 256 sequences of up to 4096 keys, 32 / 8 heads of 128
// (608 MB): 125 us, 0.72 of measured HBM; 2 of 60000 to 100000 keys, 32 / 32 heads (785
// MB): 145.5 us, 0.80; one of 700 keys: 7.8 us.  Bound by fixed latencies: some 300
// instructions a block of 16 keys (64 conversions and 64 scalings of pairs, 16 products,
// the rest the softmax and the turning of V) fill 60 % of the issue slots; the four warps
// that a scheduler has (the registers allow no more) wait for each other's results. (All
// of a batch of 256's instructions would issue in some 70 us.)  A short sequence is
// bound by its chain of latencies: lengths, line, page table, copies, products, join.
#include "kv4_attention.cuh"
#include "kv4_attention.h"
#include "launch.h"

namespace grg {

namespace {
constexpr int kDecSmsMax = 160;                   // SMs that the workspace has room for
constexpr int kDecWorkersMax = kDecSmsMax * 16;   // warps on them
constexpr int kPartialSlots = kDecWorkersMax * 2;
constexpr float kNoKey = -3e38f;  // the running maximum before any key
// What an item costs besides its blocks, in blocks (256 sequences up to 4096 keys: 4 128.8
// us, 6 125.0 us, 10 126.0 us; 64 of 2000 to 8000: 79.6, 78.5, 79.2 us; but 100 of 700, cut:
// 30.4, 32.5, 32.2 us).
constexpr int kItemCost = 6;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct DecodeParams {
  Kv4AttnArgs a;
  uint32_t* counters;  // [kDecWorkersMax], zero between calls
  float* part_o;       // [slot][8 * NT][D]
  float2* part_ml;     // [slot][8 * NT]
  int max_packed_rows; // sequences with more packed rows are not this kernel's
  uint32_t group_magic; // ceil(2^16 / group): r / group = r * magic >> 16 for r < 2^8
  unsigned long long wait_limit_ns;
  int wait_fault;
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;\n" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// D += A * B, m16n8k16, fp16 operands (common.cuh's, which the compiler may move).
__device__ __forceinline__ void mma_f16_add(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// D = A * B.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
// One half of an fp16 pair, twice (folds into the multiplication that takes it).
__device__ __forceinline__ uint32_t both_low(uint32_t a) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n mov.b32 %0, {l, l};\n}\n" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t both_high(uint32_t a) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n mov.b32 %0, {h, h};\n}\n" : "=r"(r) : "r"(a));
  return r;
}
// (a - m, b - n) * (c, d), two fp32 at a time.
__device__ __forceinline__ void sub_mul2(float& x, float& y, float a, float b, float m, float n, float c,
                                         float d) {
  asm("{\n .reg .b64 s, r, f;\n mov.b64 s, {%2, %3};\n mov.b64 r, {%4, %5};\n mov.b64 f, {%6, %7};\n"
      " sub.rn.f32x2 s, s, r;\n mul.rn.f32x2 s, s, f;\n mov.b64 {%0, %1}, s;\n}\n"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(m), "f"(n), "f"(c), "f"(d));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(a));
  return r;
}
}  // namespace

// One item: a group of packed rows of a sequence and a key head, and its keys.
struct DecItem {
  int blk0;  // first block of 16 keys
  int nb;    // blocks (1 where no row sees a key: nothing is loaded then)
  int hi;    // keys [.., hi) are seen by some row; 0: none
};
__device__ __forceinline__ int row_of(int packed, uint32_t magic) {
  return static_cast<int>((static_cast<uint32_t>(packed) * magic) >> 16);
}
template <int ROWS>
__device__ __forceinline__ DecItem dec_item(const Kv4Seq& s, int group, uint32_t magic, int rg,
                                            int window) {
  const int i0 = row_of(rg * ROWS, magic);
  const int i1 = row_of(min(s.take * group, (rg + 1) * ROWS) - 1, magic);
  const int hi = s.pos(i1) + 1, lo = s.first_key(i0, window);
  DecItem it;
  it.blk0 = lo / 16;
  it.hi = hi > lo ? hi : 0;
  it.nb = hi > lo ? (hi + 15) / 16 - it.blk0 : 1;
  return it;
}

// Warps of a CTA, CTAs of an SM and pairs of blocks in a warp's ring: as many
// warps as the registers allow (168 a thread with 12 warps, 128 with 16; 16 packed rows spill
// 312 bytes of 128 dimensions, 168 of 64, and 8 rows of 128 92), in one CTA an SM (ONE) or two.
template <int D, int NT, bool ONE>
struct DecShape {
  static constexpr int kCtas = ONE ? 1 : 2;
  static constexpr int kWarps = (D == 128 && NT == 2 ? 12 : 16) / kCtas;
  static constexpr int kStages = D == 64 ? 4 : 3;
};

template <int D, int NT, bool F16, bool ONE>
__global__ void __launch_bounds__(DecShape<D, NT, ONE>::kWarps * 32, DecShape<D, NT, ONE>::kCtas)
    lora_kv4_decode_kernel(const __grid_constant__ DecodeParams p) {
  using B = Kv4Block<D>;
  constexpr int kDecWarps = DecShape<D, NT, ONE>::kWarps, kDecThreads = kDecWarps * 32;
  constexpr int ROWS = 8 * NT;
  constexpr int KS = D / 16;              // k steps of S, and 16-dimension tiles of O
  constexpr int STAGES = DecShape<D, NT, ONE>::kStages;  // pairs of blocks in a warp's ring
  constexpr int kStage = 2 * B::kBytes;
  constexpr int kRing = STAGES * kStage;
  constexpr int PITCH = D + 4;            // floats of a row's partial in shared memory
  static_assert(kRing >= ROWS * PITCH * 4, "a warp's partial fits its ring");

  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t s_bar[kDecWarps * STAGES];
  __shared__ long long s_warp[2][kDecWarps];
  __shared__ int s_abort, s_last, s_top[kDecWarps];
  // until the rings start: units and items before each thread's sequences, and
  // the sequences themselves where there are no more than threads
  using Prefix = long long[kDecThreads + 1];
  Prefix* s_prefix = reinterpret_cast<Prefix*>(smem);
  Kv4Seq* s_seq = reinterpret_cast<Kv4Seq*>(smem + 2 * sizeof(Prefix));

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const Kv4AttnArgs& a = p.a;
  const int group = a.num_q_heads / a.num_kv_heads;
  const uint32_t bars = smem_u32(s_bar + warp * STAGES);
  if (lane == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(bars + 8 * i, 2 + (p.wait_fault ? 1 : 0));
    fence_mbar_init();
  }
  if (tid == 0) s_abort = 0;
  __syncthreads();
  const CtaAbort cta_abort{&s_abort, p.wait_limit_ns};
  pdl_wait();
  pdl_launch_dependents();

  // ---- the line of units (an item's fixed cost and its blocks) and of items, by
  // sequence: prefix sums over the threads' runs of sequences.  Up to 32 sequences
  // each warp has in its lanes (no barrier on the way: one sequence of 20 keys
  // 5.3 us so, 5.8 us by the CTA; a batch of 256, which goes by the CTA, pays 1 of 125 us for it).
  const bool few = a.num_seqs <= 32;
  const int per_thread = (a.num_seqs + kDecThreads - 1) / kDecThreads;
  auto seq_at = [&](int b) { return per_thread == 1 ? s_seq[b] : Kv4Seq::of(a, b); };
  auto groups_of = [&](const Kv4Seq& s) {  // row groups; 0: no rows, or not this kernel's
    return static_cast<long long>(s.take) * group > p.max_packed_rows ? 0
                                                                      : (s.take * group + ROWS - 1) / ROWS;
  };
  auto units_of = [&](const Kv4Seq& s, int& most) {  // of one key head
    long long n = 0;
    const int ng = groups_of(s);
    for (int rg = 0; rg < ng; ++rg) {
      const int nb = dec_item<ROWS>(s, group, p.group_magic, rg, a.window).nb;
      n += nb + kItemCost;
      most = max(most, nb);
    }
    return n;
  };
  long long mine[2] = {0, 0};
  int most = 0;  // blocks of the longest item
  Kv4Seq own_seq{};  // the lane's, of few
  for (int i = 0; i < per_thread; ++i) {
    const int b = (few ? lane : tid) * per_thread + i;
    if (b < a.num_seqs) {
      const Kv4Seq s = Kv4Seq::of(a, b);
      if (few) own_seq = s;
      else if (per_thread == 1) s_seq[b] = s;
      if (s.odd && blockIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadLength);
      mine[0] += units_of(s, most) * a.num_kv_heads;
      mine[1] += static_cast<long long>(groups_of(s)) * a.num_kv_heads;
    }
  }
  long long run[2] = {mine[0], mine[1]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const long long v = __shfl_up_sync(0xffffffffu, run[i], o);
      if (lane >= o) run[i] += v;
    }
  most = __reduce_max_sync(0xffffffffu, most);
  long long all[2] = {0, 0};
  if (few) {
#pragma unroll
    for (int i = 0; i < 2; ++i) all[i] = __shfl_sync(0xffffffffu, run[i], 31);
  } else {
    if (lane == 31) s_warp[0][warp] = run[0], s_warp[1][warp] = run[1], s_top[warp] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) most = max(most, s_top[w]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      long long before = 0;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        if (w < warp) before += s_warp[i][w];
        all[i] += s_warp[i][w];
      }
      s_prefix[i][tid] = before + run[i] - mine[i];
      if (tid == 0) s_prefix[i][kDecThreads] = all[i];
    }
    __syncthreads();
  }
  if (all[0] == 0) return;

  // ---- who takes what.  A cut item costs its join (partials to L2, a counter,
  // and back: about 6 us on the way of the last), so items stay whole where the
  // longest runs over a worker's fair share by less than that: 160 blocks of a CTA
  // that has one item, 40 of a CTA that has two, 16 of a warp.  (48 windows of
  // 2048 keys, 30 rows of 64: 20.2 us whole, 36.1 cut; 150 sequences of 1500 to 2000
  // keys, two items a CTA: 42.5 and 49.3 us.  Three are cut, which an item's cost of 4
  // called for; with 6, 100 sequences of 700 keys take 31.1 us whole and 32.5 cut.)
  // A CTA goes before a warp, which takes 0.6 us a block: 8 items of 200 keys 5.7 and
  // 13.3 us, two items a CTA, 100 to 200 keys, 12.8 and 18.2 us; 512 sequences of 20 to
  // 100 keys, one head, 13.3 and 12.1 us.  Else the line of units is cut into equal runs, of warps, or of
  // CTAs where an item would span over 8 warps' runs (20 sequences of 2000 to 5000
  // keys, 16 rows).
  // (Few divisions: they are on every call's way.)
  const long long ctas = gridDim.x, warps_all = ctas * kDecWarps;
  const int cta_items = all[1] <= ctas ? 1 : all[1] <= 2 * ctas ? 2 : 3;
  const bool whole_cta = (cta_items == 1 && (most - 160ll) * ctas <= all[0]) ||
                         (cta_items == 2 && most > 8 && (2ll * most - 40) * ctas <= all[0]);
  bool whole = whole_cta, team = whole_cta;
  long long per = cta_items;
  if (!whole_cta) {
    const long long per_warp = max(quotient(all[0] + warps_all - 1, warps_all), 2ll * kItemCost);
    const long long warp_items = quotient(all[1] + warps_all - 1, warps_all);
    whole = warp_items * (most + kItemCost) <= per_warp + 16;
    team = !whole && all[0] > 8 * per_warp * all[1];
    per = whole ? warp_items
                : team ? max(quotient(all[0] + ctas - 1, ctas), 2ll * kDecWarps) : per_warp;
  }
  const long long total = whole ? all[1] : all[0];  // items are the units where they stay whole
  const int worker = team ? blockIdx.x : blockIdx.x * kDecWarps + warp;
  const int TW = team ? kDecWarps : 1, wt = team ? warp : 0;
  auto team_sync = [&]() {
    if (team) __syncthreads(); else __syncwarp();
  };
  unsigned char* ring = smem + warp * kRing;
  const uint32_t ring_u = smem_u32(ring);
  float* own = reinterpret_cast<float*>(ring);  // the warp's partial, once its ring is idle
  int stage_in = 0, stage_out = 0;              // where the next copy goes, and comes from
  uint32_t phase = 0;                           // of stage_out's barrier

  const long long u0 = worker * per, u_end = min(u0 + per, total);
  const int cost = whole ? 0 : kItemCost;
  auto run_of = [&](long long x) { return static_cast<int>(quotient(x, per)); };  // the worker of place x
  // the part of an item that this worker has: blocks [o, o + take) of the item
  // whose place in the line is [at, at + cost + nb)
  int b = 0, rg = 0, h = 0, o = 0, take = 0;
  int at = 0;  // from u0
  const int run_len = static_cast<int>(u_end - u0);
  Kv4Seq seq;
  DecItem item;
  auto set_take = [&]() {
    take = whole ? item.nb : min(item.nb, run_len - at - cost) - o;
  };
  if (u0 < u_end) {
    long long off;
    if (few) {
      const long long begins = whole ? run[1] - mine[1] : run[0] - mine[0];
      b = __popc(__ballot_sync(0xffffffffu, begins <= u0)) - 1;
      off = u0 - __shfl_sync(0xffffffffu, begins, b);
      seq.q0 = __shfl_sync(0xffffffffu, own_seq.q0, b);
      seq.rows = __shfl_sync(0xffffffffu, own_seq.rows, b);
      seq.take = __shfl_sync(0xffffffffu, own_seq.take, b);
      seq.kv = __shfl_sync(0xffffffffu, own_seq.kv, b);
    } else {
      const long long* prefix = s_prefix[whole ? 1 : 0];
      const int lo = last_not_past<kDecWarps>(prefix, u0, lane);
      int ignored = 0;
      off = u0 - prefix[lo];
      for (b = lo * per_thread;; ++b) {
        seq = seq_at(b);
        const long long n = (whole ? groups_of(seq) : units_of(seq, ignored)) * a.num_kv_heads;
        if (off < n) break;
        off -= n;
      }
    }
    int size;
    while (true) {
      item = dec_item<ROWS>(seq, group, p.group_magic, rg, a.window);
      size = whole ? 1 : item.nb + cost;
      if (off < static_cast<long long>(size) * a.num_kv_heads) break;
      off -= static_cast<long long>(size) * a.num_kv_heads;
      ++rg;
    }
    h = static_cast<int>(quotient(off, size));
    off -= static_cast<long long>(h) * size;
    at = -static_cast<int>(off);
    o = max(static_cast<int>(off) - cost, 0);
    set_take();
  }
  auto advance = [&]() -> bool {  // to the worker's next part
    at += whole ? 1 : cost + item.nb;
    if (at >= run_len) return false;
    o = 0;
    if (++h == a.num_kv_heads) {
      h = 0;
      ++rg;
      while (rg >= groups_of(seq)) {
        rg = 0;
        seq = Kv4Seq::of(a, ++b);
      }
      item = dec_item<ROWS>(seq, group, p.group_magic, rg, a.window);
    }
    set_take();
    return take > 0;
  };
  if (!few) {  // the rings may start
    fence_proxy_async();
    __syncthreads();
  }
  if (take <= 0) return;  // a whole team or a lone warp

  // ---- a part's copies: pairs of blocks 2 q, 2 q + 1 of it, q = wt + TW k for this warp
  const int page_blocks = a.page_size / 16;
  const int32_t* table = nullptr;
  int first_blk = 0, part_take = 0, part_h = 0, np = 0, issued = 0;
  unsigned long long now = 0;
  bool hole = false;  // some page (of those looked up so far) is not in the cache
  // pairs [k_open, k_open + k_shut) of a part need no mask: both blocks exist, every row
  // sees every key
  int k_open = 0, k_shut = 0;
  auto block_at = [&](int blk) -> const unsigned char* {  // null: its page is not in the cache
    const int pg = blk / page_blocks;
    const int page = __ldg(table + pg);
    if (page < 0 || page >= a.num_pages) return nullptr;
    return a.cache + ((static_cast<long long>(page) * a.num_kv_heads + part_h) * page_blocks +
                      (blk - pg * page_blocks)) * B::kBytes;
  };
  // block addresses: 16 pairs at a time, lane l holds block l & 1 of pair l / 2 (null: not there)
  auto addresses = [&](int k0) -> unsigned long long {
    const int i = 2 * (wt + TW * (k0 + (lane >> 1))) + (lane & 1);
    const unsigned char* x = i < part_take ? block_at(first_blk + i) : nullptr;
    if (__any_sync(0xffffffffu, i < part_take && !x)) {
      hole = true;
      if (lane == 0 && a.status) atomicOr(a.status, kStatusBadSlot);
    }
    return reinterpret_cast<unsigned long long>(x);
  };
  auto issue = [&](int k) {  // by the two lanes that hold pair k's addresses
    if ((k & 15) == 0 && k > 0) {
      now = addresses(k);
      if (hole) k_shut = 0;  // these pairs are scored after this
    }
    if ((lane >> 1) == (k & 15)) {
      const uint32_t bar = bars + 8 * stage_in;
      mbar_arrive_expect_tx(bar, now ? B::kBytes : 0);
      if (now)
        bulk_g2s(ring_u + stage_in * kStage + (lane & 1) * B::kBytes,
                 reinterpret_cast<const void*>(now), B::kBytes, bar);
    }
    if (++stage_in == STAGES) stage_in = 0;
  };
  auto begin = [&]() {
    first_blk = item.blk0 + o, part_take = take, part_h = h;
    table = a.page_table + static_cast<long long>(b) * a.table_stride;
    np = item.hi > 0 && !p.wait_fault ? ((take + 1) / 2 - wt + TW - 1) / TW : (p.wait_fault ? 1 : 0);
    hole = false;
    // After a wait has given up no part begins (those under way go on while their copies
    // arrive), so every barrier that is drained has a copy on its way.
    if (__any_sync(0xffffffffu, cta_abort.raised())) np = 0;
    now = np > 0 && !p.wait_fault ? addresses(0) : 0;
    for (issued = 0; issued < min(np, STAGES); ++issued) issue(issued);
  };
  // this thread's share of the rows' queries (D / 4 dimensions of row g of each 8), which
  // a first part asks for before its pages are looked up
  uint4 raw_q[NT][KS / 2];
  auto load_q = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = rg * ROWS + nt * 8 + g;
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) raw_q[nt][i] = make_uint4(0, 0, 0, 0);
      if (r < seq.take * group) {
        const int i = row_of(r, p.group_magic);
        const uint16_t* src = a.q + (seq.q0 + i) * a.q_stride + (h * group + r - i * group) * D +
                              t4 * (D / 4);
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) raw_q[nt][i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
      }
    }
  };
  load_q();
  begin();

  while (true) {
    const int packed = seq.take * group;  // packed rows of the sequence
    const int row0 = rg * ROWS;
    const int live_rows = min(packed - row0, ROWS);

    // ---- the rows' queries as B fragments, in fp16, and what undoes their factor
    uint32_t qf[NT][KS][2];
    float cf[NT][2];
    int pos[NT][2], lo[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float v[KS * 4], top = 0.0f;
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {
        const uint32_t x[4] = {raw_q[nt][i].x, raw_q[nt][i].y, raw_q[nt][i].z, raw_q[nt][i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = unpack_t<F16>(x[k]);
          v[8 * i + 2 * k] = f.x, v[8 * i + 2 * k + 1] = f.y;
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      float up, down;
      row_factor(top, up, down);
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        qf[nt][j][0] = pack_f16x2(v[4 * j] * up, v[4 * j + 1] * up);
        qf[nt][j][1] = pack_f16x2(v[4 * j + 2] * up, v[4 * j + 3] * up);
      }
      // the thread's columns of S and O are rows 2 t4 and 2 t4 + 1 of the tile
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        cf[nt][c] = score_factor(__shfl_sync(0xffffffffu, down, (2 * t4 + c) * 4), a.score_scale * kLog2e);
        const int rr = row_of(min(row0 + nt * 8 + 2 * t4 + c, packed - 1), p.group_magic);
        pos[nt][c] = seq.pos(rr);
        lo[nt][c] = seq.first_key(rr, a.window);
      }
    }
    const int pos_min = seq.pos(row_of(row0, p.group_magic)), pos_max = item.hi - 1;
    const int lo_max = seq.first_key(row_of(row0 + live_rows - 1, p.group_magic), a.window);

    float acc[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) m[nt][c] = kNoKey, l[nt][c] = 0.0f;
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[nt][i][c] = 0.0f;
    }
    bool poison = false;  // a NaN scale of V among keys that some rows must not see

    {
      const int last = min(min((pos_min + 1) / 16 - first_blk, part_take), 1 << 27);  // blocks all rows see
      const int first = max((lo_max + 15) / 16 - first_blk, 0);
      const int q1 = last / 2, q0 = (first + 1) / 2;  // pairs
      k_open = q0 <= wt ? 0 : (q0 - wt + TW - 1) / TW;
      k_shut = hole || q1 <= wt ? 0 : max((q1 - wt + TW - 1) / TW - k_open, 0);
    }

    // key of this thread's S rows g and g + 8 (parities alternate: no bank conflicts)
    const int kr = g ^ ((g >> 1) & 1);
    int k = 0;
    for (; k < np; ++k) {
      {
        bool ok = mbar_try_wait(bars + 8 * stage_out, phase);
        if (!ok) ok = cta_abort.wait(bars + 8 * stage_out, phase);
        if (!__all_sync(0xffffffffu, ok)) break;
      }
      const unsigned char* stage = ring + stage_out * kStage;
      const bool masked = static_cast<uint32_t>(k - k_open) >= static_cast<uint32_t>(k_shut);
      const int i0 = 2 * (wt + TW * k);       // the pair's first block in the part
      const int tok = 16 * (first_blk + i0);  // and its first key
      uint32_t have = 3u;
      if (masked) {
        if (i0 + 1 >= part_take) have = 1u;
        if (hole) {
          if (!block_at(first_blk + i0)) have &= 2u;
          if (i0 + 1 < part_take && !block_at(first_blk + i0 + 1)) have &= 1u;
        }
      }

      float sc[NT][2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const unsigned char* blk = stage + x * B::kBytes;
        uint32_t ca[D / 32], cb[D / 32];
        uint32_t sa[2], sb[2];  // scales of the thread's first and second 16 dimensions
        if constexpr (D == 128) {
          const uint4 va = *reinterpret_cast<const uint4*>(blk + kr * 64 + 16 * t4);
          const uint4 vb = *reinterpret_cast<const uint4*>(blk + (kr + 8) * 64 + 16 * t4);
          ca[0] = va.x, ca[1] = va.y, ca[2] = va.z, ca[3] = va.w;
          cb[0] = vb.x, cb[1] = vb.y, cb[2] = vb.z, cb[3] = vb.w;
          const uint32_t ha = e4m3x2_to_f16(
              *reinterpret_cast<const uint16_t*>(blk + B::kKScale + kr * 8 + 2 * t4));
          const uint32_t hb = e4m3x2_to_f16(
              *reinterpret_cast<const uint16_t*>(blk + B::kKScale + (kr + 8) * 8 + 2 * t4));
          sa[0] = both_low(ha), sa[1] = both_high(ha);
          sb[0] = both_low(hb), sb[1] = both_high(hb);
        } else {
          const uint2 va = *reinterpret_cast<const uint2*>(blk + kr * 32 + 8 * t4);
          const uint2 vb = *reinterpret_cast<const uint2*>(blk + (kr + 8) * 32 + 8 * t4);
          ca[0] = va.x, ca[1] = va.y, cb[0] = vb.x, cb[1] = vb.y;
          const uint32_t ha = e4m3x2_to_f16(blk[B::kKScale + kr * 4 + t4]);
          const uint32_t hb = e4m3x2_to_f16(blk[B::kKScale + (kr + 8) * 4 + t4]);
          sa[0] = sa[1] = both_low(ha);
          sb[0] = sb[1] = both_low(hb);
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t ha[4], hb[4];
          e2m1x8_to_f16(ca[w], ha);
          e2m1x8_to_f16(cb[w], hb);
          const uint32_t fa = sa[w / 2], fb = sb[w / 2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t frag[4] = {hmul2(ha[2 * j], fa), hmul2(hb[2 * j], fb),
                                      hmul2(ha[2 * j + 1], fa), hmul2(hb[2 * j + 1], fb)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (w == 0 && j == 0) mma_f16_first(sc[nt][x], frag, qf[nt][0][0], qf[nt][0][1]);
              else mma_f16_add(sc[nt][x], frag, qf[nt][2 * w + j][0], qf[nt][2 * w + j][1]);
            }
          }
        }
      }

      // ---- probabilities against the running reference m, which moves only when
      // some score passes it by 2^6
      if (masked) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int j = tok + 16 * x + kr + 8 * (c >> 1);
              if (j > pos[nt][c & 1] || j < lo[nt][c & 1] || !((have >> x) & 1u))
                sc[nt][x][c] = -INFINITY;
            }
      }
      bool move = false;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mx[nt][c] = fmaxf(fmaxf(sc[nt][0][c], sc[nt][0][c + 2]),
                            fmaxf(sc[nt][1][c], sc[nt][1][c + 2]));
          move = move || (mx[nt][c] - m[nt][c]) * cf[nt][c] > 6.0f;
        }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v = mx[nt][c];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            const float to = fmaxf(m[nt][c], v);
            const float f = exp2_approx((m[nt][c] - to) * cf[nt][c]);
            m[nt][c] = to;
            l[nt][c] *= f;
#pragma unroll
            for (int i = 0; i < KS; ++i) acc[nt][i][c] *= f, acc[nt][i][c + 2] *= f;
          }
      }
      uint32_t pb[NT][2][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float p0, p1, p2, p3;
          sub_mul2(p0, p1, sc[nt][x][0], sc[nt][x][1], m[nt][0], m[nt][1], cf[nt][0], cf[nt][1]);
          sub_mul2(p2, p3, sc[nt][x][2], sc[nt][x][3], m[nt][0], m[nt][1], cf[nt][0], cf[nt][1]);
          p0 = exp2_approx(p0), p1 = exp2_approx(p1), p2 = exp2_approx(p2), p3 = exp2_approx(p3);
          l[nt][0] += p0 + p2;
          l[nt][1] += p1 + p3;
          pb[nt][x][0] = transpose8x8(pack_f16x2(p0, p1));
          pb[nt][x][1] = transpose8x8(pack_f16x2(p2, p3));
        }
      }

      // ---- O += V^T P
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const unsigned char* blk = stage + x * B::kBytes;
        const int r0 = 2 * t4 ^ (t4 & 1), r1 = (2 * t4 + 1) ^ (t4 & 1);  // keys of k = 2 t4, 2 t4 + 1
        const unsigned char* scales = blk + B::kVScale + (D == 128 ? g : g / 2);
        uint32_t e0 = scales[r0 * (D / 16)], e1 = scales[r1 * (D / 16)];
        uint32_t e2 = scales[(r0 + 8) * (D / 16)], e3 = scales[(r1 + 8) * (D / 16)];
        if (masked) {
          // keys that no row sees may hold anything; a NaN scale among the
          // others must not reach the rows that do not see its key
          auto clean = [&](uint32_t& e, int r) {
            const int j = tok + 16 * x + r;
            if (j > pos_max || !((have >> x) & 1u)) e = 0;
            if ((e & 0x7Fu) == 0x7Fu) poison = true, e = 0;
          };
          clean(e0, r0), clean(e1, r1), clean(e2, r0 + 8), clean(e3, r1 + 8);
        }
        const uint32_t s01 = e4m3x2_to_f16(prmt(e0, e1, 0x40)), s23 = e4m3x2_to_f16(prmt(e2, e3, 0x40));
        constexpr int W = D / 64;  // words of a key's dimensions
        uint32_t c0[W], c1[W], c2[W], c3[W];
        auto load = [&](uint32_t (&c)[W], int r) {
          const unsigned char* at = blk + B::kV + r * B::kCodeRow + 4 * W * g;
          if constexpr (W == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(at);
            c[0] = v.x, c[1] = v.y;
          } else {
            c[0] = *reinterpret_cast<const uint32_t*>(at);
          }
        };
        load(c0, r0), load(c1, r1), load(c2, r0 + 8), load(c3, r1 + 8);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          // byte i of a word holds dimensions 2 i, 2 i + 1 of one key; of the
          // pairs below, one dimension of two keys
          constexpr uint32_t L = 0x0F0F0F0Fu;
          uint32_t ev[4], od[4], ev2[4], od2[4];
          e2m1x8_to_f16((c0[w] & L) | ((c1[w] << 4) & ~L), ev);
          e2m1x8_to_f16(((c0[w] >> 4) & L) | (c1[w] & ~L), od);
          e2m1x8_to_f16((c2[w] & L) | ((c3[w] << 4) & ~L), ev2);
          e2m1x8_to_f16(((c2[w] >> 4) & L) | (c3[w] & ~L), od2);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t frag[4] = {hmul2(ev[i], s01), hmul2(od[i], s01), hmul2(ev2[i], s23),
                                      hmul2(od2[i], s23)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16_add(acc[nt][4 * w + i], frag, pb[nt][x][0], pb[nt][x][1]);
          }
        }
      }
      __syncwarp();
      if (++stage_out == STAGES) stage_out = 0, phase ^= 1;
      if (issued < np) issue(issued++);
    }
    if (k < np)  // gave up: what is still on its way lands before the ring is left
      for (; k < issued; ++k) {
        mbar_drain(bars + 8 * stage_out, phase, p.wait_limit_ns);
        if (++stage_out == STAGES) stage_out = 0, phase ^= 1;
      }

    // ---- join: sums over the lanes that share a row; m in units of log2 from here on
    // (finite: no difference of two is a NaN)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[nt][c] = fmaxf(m[nt][c] * cf[nt][c], kNoKey);
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 4);
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 8);
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 16);
      }
    if (__any_sync(0xffffffffu, poison)) {
      // rare: which of its 16 dimensions' scales are NaN at keys a row sees
      for (int i = 0; i < part_take; ++i) {
        if (TW > 1 && (i / 2) % TW != wt) continue;
        const int blk = first_blk + i;
        const unsigned char* at = block_at(blk);
        if (!at) continue;
        at += B::kVScale + (D == 128 ? g : g / 2);
        for (int r = 0; r < 16; ++r)
          if ((at[r * (D / 16)] & 0x7F) == 0x7F)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                if (blk * 16 + r <= pos[nt][c] && blk * 16 + r >= lo[nt][c])
#pragma unroll
                  for (int q = 0; q < KS; ++q)
                    acc[nt][q][c] = acc[nt][q][c + 2] = __uint_as_float(0x7FC00000u);
      }
    }

    // ---- the next part's copies may start: this one needs its ring no more (but
    // for a team's join); then this part's rows go out
    const int out_h = h, out_q0 = seq.q0, nb = item.nb;
    const bool all_of_it = take == item.nb;
    const int slot = worker * 2 + (o == 0 ? 1 : 0);
    const int begins = at + cost;
    const bool more = advance();
    if (more && !team) begin();
    // where row r goes: its place in out (with what turns sums into values) or in
    // the partials
    struct RowOut {
      uint16_t* out;
      float* part;
      float inv;
    };
    auto open_row = [&](int r, bool whole_row, float top, float sum, bool writer) {
      RowOut w{nullptr, nullptr, 0.0f};
      if (whole_row) {
        const int pr = row0 + r, i = row_of(pr, p.group_magic), head = out_h * group + pr - i * group;
        const long long t = out_q0 + i;
        w.out = cta_abort.raised() ? nullptr : a.out + t * a.out_stride + head * D;
        w.inv = sum == 0.0f ? 0.0f : a.v_scale / sum;
        if (writer && w.out && a.lse)
          a.lse[t * a.num_q_heads + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
      } else {
        w.part = p.part_o + static_cast<long long>(slot * ROWS + r) * D;
        if (writer) p.part_ml[slot * ROWS + r] = make_float2(top, sum);
      }
      return w;
    };
    auto put4 = [&](const RowOut& w, int d, float4 v) {
      if (w.part) {
        *reinterpret_cast<float4*>(w.part + d) = v;
      } else if (w.out) {
        uint2 o2;
        o2.x = pack_t<F16>(v.x * w.inv, v.y * w.inv);
        o2.y = pack_t<F16>(v.z * w.inv, v.w * w.inv);
        *reinterpret_cast<uint2*>(w.out + d) = o2;
      }
    };
    // Joins the team's warps' rows, [row][D] and (m, l) in each warp's ring, and
    // hands them on; 4 dimensions a thread.
    auto join = [&](bool whole_rows) {
      __syncthreads();
      for (int i = tid; i < live_rows * (D / 4); i += kDecThreads) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        const float* base = reinterpret_cast<const float*>(smem) + r * PITCH;
        float top = kNoKey;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) top = fmaxf(top, base[w * (kRing / 4) + D]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          const float* part = base + w * (kRing / 4);
          const float2 ml = *reinterpret_cast<const float2*>(part + D);
          const float f = exp2_approx(ml.x - top);
          const float4 x = *reinterpret_cast<const float4*>(part + d);
          sum += ml.y * f;
          v.x += x.x * f, v.y += x.y * f, v.z += x.z * f, v.w += x.w * f;
        }
        put4(open_row(r, whole_rows, top, sum, d == 0), d, v);
      }
    };
    // This warp's rows: straight on where it works alone, else through the join.
    auto hand_on = [&](bool whole_rows) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = nt * 8 + 2 * t4 + c;
          if (r >= live_rows) continue;
          RowOut w{nullptr, own + r * PITCH, 0.0f};
          if (!team) w = open_row(r, whole_rows, m[nt][c], l[nt][c], g == 0);
          else if (g == 0) *reinterpret_cast<float2*>(own + r * PITCH + D) = make_float2(m[nt][c], l[nt][c]);
#pragma unroll
          for (int i = 0; i < KS; i += 2)
            put4(w, (D / 8) * g + 2 * i, make_float4(acc[nt][i][c], acc[nt][i][c + 2], acc[nt][i + 1][c],
                                                     acc[nt][i + 1][c + 2]));
        }
      if (team) join(whole_rows);
    };
    if (all_of_it) {
      hand_on(true);
    } else {
      const int w0 = run_of(u0 + begins), w1 = run_of(u0 + begins + nb - 1);
      hand_on(false);
      team_sync();
      int last = 0;
      if (wt == 0 && lane == 0) {
        uint32_t seen;  // releases what the barrier above has gathered, acquires the others'
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;\n"
                     : "=r"(seen)
                     : "l"(p.counters + w0)
                     : "memory");
        last = seen == static_cast<uint32_t>(w1 - w0);
        if (last) p.counters[w0] = 0;
        if (team) s_last = last;
      }
      if (team) {
        __syncthreads();
        last = s_last;
      } else {
        last = __shfl_sync(0xffffffffu, last, 0);
      }
      if (last) {
        // every run of the item is there: each warp sums its share of them, in
        // run order, 32 at a time; a lane holds D / 32 dimensions of every row
        const int n = (w1 - w0 + TW - wt) / TW;  // runs of this warp: wt, wt + TW, ...
        constexpr int E = D / 32, RB = 4, JB = D == 64 ? 4 : 2;  // rows and runs loaded together
        auto slot_of = [&](int j) {
          const int i = wt + TW * j;
          return ((static_cast<long long>(w0) + i) * 2 + (i == 0 ? 1 : 0)) * ROWS;
        };
        for (int r0 = 0; r0 < live_rows; r0 += RB) {
          float v[RB][E] = {}, top[RB], sum[RB] = {};
#pragma unroll
          for (int r = 0; r < RB; ++r) top[r] = kNoKey;
          for (int j0 = 0; j0 < n; j0 += 32) {
            float2 ml[RB];
            const float2* src = p.part_ml + slot_of(min(j0 + lane, n - 1)) + r0;
#pragma unroll
            for (int r = 0; r < RB; ++r)
              ml[r] = r0 + r < live_rows && j0 + lane < n ? __ldcg(src + r) : make_float2(kNoKey, 0.0f);
            const int some = min(32, n - j0);
            float x[JB][RB][E];
            auto fetch = [&](int j) {
#pragma unroll
              for (int i = 0; i < JB; ++i) {
                const float* o_src = p.part_o + (slot_of(min(j0 + j + i, n - 1)) + r0) * D + lane * E;
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                  const bool in = r0 + r < live_rows && j + i < some;
                  if constexpr (E == 4) {
                    const float4 q = in ? __ldcg(reinterpret_cast<const float4*>(o_src + r * D))
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                    x[i][r][0] = q.x, x[i][r][1] = q.y, x[i][r][2] = q.z, x[i][r][3] = q.w;
                  } else {
                    const float2 q = in ? __ldcg(reinterpret_cast<const float2*>(o_src + r * D))
                                        : make_float2(0.f, 0.f);
                    x[i][r][0] = q.x, x[i][r][1] = q.y;
                  }
                }
              }
            };
            fetch(0);  // on its way together with the maxima
#pragma unroll
            for (int r = 0; r < RB; ++r) {
              float to = ml[r].x;
#pragma unroll
              for (int s = 16; s; s >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, s));
              to = fmaxf(to, top[r]);
              const float f = exp2_approx(top[r] - to);
              top[r] = to;
              sum[r] *= f;
#pragma unroll
              for (int e = 0; e < E; ++e) v[r][e] *= f;
              ml[r].x = exp2_approx(ml[r].x - to);
            }
            for (int j = 0; j < some; j += JB) {
#pragma unroll
              for (int i = 0; i < JB; ++i)
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                  const float f = __shfl_sync(0xffffffffu, ml[r].x, (j + i) & 31);
                  const float s = __shfl_sync(0xffffffffu, ml[r].y, (j + i) & 31);
                  sum[r] += j + i < some ? s * f : 0.0f;
#pragma unroll
                  for (int e = 0; e < E; ++e) v[r][e] += j + i < some ? x[i][r][e] * f : 0.0f;
                }
              if (j + JB < some) fetch(j + JB);
            }
          }
#pragma unroll
          for (int r = 0; r < RB; ++r) {
            if (r0 + r >= live_rows) break;
            if (team) {
              float* row = own + (r0 + r) * PITCH;
#pragma unroll
              for (int e = 0; e < E; ++e) row[lane * E + e] = v[r][e];
              if (lane == 0) *reinterpret_cast<float2*>(row + D) = make_float2(top[r], sum[r]);
            } else {
              const RowOut w = open_row(r0 + r, true, top[r], sum[r], lane == 0);
              if (w.out)
#pragma unroll
                for (int e = 0; e < E; e += 2)
                  *reinterpret_cast<uint32_t*>(w.out + lane * E + e) =
                      pack_t<F16>(v[r][e] * w.inv, v[r][e + 1] * w.inv);
            }
          }
        }
        if (team) join(true);
      }
    }
    if (!more) break;
    load_q();
    if (team) {
      fence_proxy_async();  // the rings' next writes are bulk copies
      __syncthreads();
      begin();
    }
  }
  if (lane == 0 && cta_abort.raised() && a.status) atomicOr(a.status, kStatusTimeout);
}

namespace {
template <int D, int NT, bool F16, bool ONE>
int run_decode(const DecodeParams& q, int sms, cudaStream_t stream) {
  using S = DecShape<D, NT, ONE>;
  DecodeParams p = q;
  const void* fn = reinterpret_cast<const void*>(lora_kv4_decode_kernel<D, NT, F16, ONE>);
  const size_t smem = static_cast<size_t>(S::kWarps) * S::kStages * 2 * Kv4Block<D>::kBytes;
  if (ensure_smem_attr(fn, smem) != 0) return -6;
  return launch_pdl(fn, dim3(S::kCtas * sms), dim3(S::kWarps * 32), smem, stream, 0, &p);
}
constexpr size_t kCounterBytes = kDecWorkersMax * 4;
}  // namespace

size_t kv4_decode_counter_bytes() { return kCounterBytes; }
size_t kv4_decode_partial_bytes(int rows, int head_dim) {
  return static_cast<size_t>(kPartialSlots) * rows * (head_dim * 4 + 8);
}

int launch_kv4_decode(const Kv4AttnArgs& a, int max_packed_rows, size_t counters_at, bool f16,
                      cudaStream_t stream) {
  const int group = a.num_q_heads / a.num_kv_heads;
  const bool wide = static_cast<long long>(a.max_q_len) * group > 8;
  DecodeParams p;
  p.a = a;
  char* w = static_cast<char*>(a.workspace) + counters_at;
  const int rows = wide ? 16 : 8;
  p.counters = reinterpret_cast<uint32_t*>(w);
  p.part_o = reinterpret_cast<float*>(w + kCounterBytes);
  p.part_ml = reinterpret_cast<float2*>(w + kCounterBytes +
                                        static_cast<size_t>(kPartialSlots) * rows * a.head_dim * 4);
  p.max_packed_rows = max_packed_rows;
  p.group_magic = (65536u + group - 1) / group;
  p.wait_fault = wait_fault() ? 1 : 0;
  p.wait_limit_ns = p.wait_fault ? kTestWaitLimitNs : kWaitLimitNs;
  const int sms = min(device_sm_count(), kDecSmsMax);
  if (sms <= 0) return -6;
  if (a.head_dim == 64)
    return wide ? (f16 ? run_decode<64, 2, true, false>(p, sms, stream)
                       : run_decode<64, 2, false, false>(p, sms, stream))
                : (f16 ? run_decode<64, 1, true, false>(p, sms, stream)
                       : run_decode<64, 1, false, false>(p, sms, stream));
  if (!wide)
    return f16 ? run_decode<128, 1, true, false>(p, sms, stream)
               : run_decode<128, 1, false, false>(p, sms, stream);
  // Where there can be no more items than SMs, CTAs of all of an SM's warps: 10
  // sequences of 1000 to 1500 keys, 8 key heads, 16 rows: 14.3 us so, 22.0 us by two an SM;
  // 60 of 500, 4 key heads: 19.4 us by one, 14.0 us by two.
  const long long packed = min(static_cast<long long>(a.max_q_len) * group,
                               static_cast<long long>(max_packed_rows));
  if ((packed + 15) / 16 * a.num_seqs * a.num_kv_heads <= sms)
    return f16 ? run_decode<128, 2, true, true>(p, sms, stream)
               : run_decode<128, 2, false, true>(p, sms, stream);
  return f16 ? run_decode<128, 2, true, false>(p, sms, stream)
             : run_decode<128, 2, false, false>(p, sms, stream);
}

}  // namespace grg
