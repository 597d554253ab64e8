// The key weights of sequences with many query rows (chunks of prefill, long paths), on the
// 5th-generation tensor cores.
//
// An item is 256 keys of one key head, as two tiles of 128, against all packed rows (row x head
// of the key head) that see one of them, 128 at a time:
//   S_t = K_t Q^T (M = 128 keys, N = rows),  w[key] += sum over rows of 2^(S c - lse log2 e)
// Keys are the lanes of TMEM, so a key's sum is one thread's: nothing is exchanged, no key's
// sum is cut, and each is formed in the rows' order.  K stays in shared memory while
// the rows pass by.  It is widened to q's own 16-bit type: a code times its e4m3 scale has at
// most six significant bits, which bf16 holds too, so that q is copied as it is and c is
// the same for all rows.
//
// Warp roles (16 warps of 128 registers, one CTA per SM, persistent):
//  - warps 0-3 and 4-7: the sums of tile 0 and 1; a thread owns a key
//  - warps 8-11: widen K into swizzled operand tiles, an item ahead of the products
//  - warps 12-14: copy the rows of q and their logarithms, two row tiles deep
//  - warp 15: issues the products; S is double-buffered in TMEM
// Work: items by the number of their row tiles, most first, dealt out to the CTAs to and fro;
// where they are too many to sort (over kTcPairs pairs of sequence and keys) in their own order.
#include "kv4_weights.cuh"
#include "launch.h"

namespace grg {

namespace {
constexpr int kTcThreads = 512, kTcWarps = kTcThreads / 32;
constexpr int kTcRowThreads = 96;  // that copy rows
constexpr int kTcKeys = 256;   // keys of an item
constexpr int kTcRows = 128;   // packed rows of a tile
constexpr int kTcPairs = 512;  // (sequence, keys) pairs that are sorted
constexpr int kTcAhead = 4;    // row tiles' logarithms kept
constexpr float kTcLog2e = 1.4426950408889634f;

struct TcParams {
  Kv4WeightsArgs a;
  int max_packed_rows;  // sequences with no more packed rows are not this kernel's
  unsigned long long wait_limit_ns;
  int wait_fault;
};

struct TcShared {
  uint64_t q_full[2], q_empty[2];  // by row tile: the rows are there; their products are done
  uint64_t l_full[kTcAhead];       // and their logarithms
  uint64_t k_full[2], k_empty[2];  // by item
  uint64_t s_full[2], s_empty[2];  // by row tile
  uint64_t drain;
  __align__(16) float neg[kTcAhead][kTcRows];  // -lse log2 e of a tile's rows, -infinity: adds nothing
  int odd[kTcAhead];                           // a row that exists adds nothing
  uint32_t taddr;
  int abort;
  int warp_sum[kTcWarps];
  long long warp_long[kTcWarps];
  long long prefix[kTcThreads + 1];  // pairs before a thread's sequences
  int pair_b[kTcPairs], pair_kt[kTcPairs], pair_tiles[kTcPairs];
  int sorted[kTcPairs];
};

// An item: its keys [256 kt, ...) and the packed rows [row0, row0 + rows) that see one of them.
struct TcItem {
  int b, h, kt;
  WeightSeq seq;
  int row0, rows;
  __device__ __forceinline__ int tiles() const { return (rows + kTcRows - 1) / kTcRows; }
};
__device__ __forceinline__ bool tc_mine(const WeightSeq& s, int group, int max_packed_rows) {
  return s.rows > 0 && static_cast<long long>(s.take) * group > max_packed_rows;
}
// Key tiles of a sequence: [first, first + count).
__device__ __forceinline__ int tc_first(const WeightSeq& s, int window) { return s.first_key(0, window) / kTcKeys; }
__device__ __forceinline__ int tc_count(const WeightSeq& s, int window) {
  return max((s.end + kTcKeys - 1) / kTcKeys - tc_first(s, window), 0);
}
__device__ __forceinline__ void tc_rows(const WeightSeq& s, int kt, int group, int window, int& row0, int& rows) {
  const int before = s.kv - s.rows;
  const int key0 = kt * kTcKeys, key1 = min(key0 + kTcKeys, s.end) - 1;
  const int i0 = max(key0 - before, 0);
  long long i1 = s.take - 1;
  if (window > 0) i1 = min(i1, static_cast<long long>(key1) + window - 1 - before);
  row0 = i0 * group;
  rows = i1 >= i0 ? static_cast<int>(i1 - i0 + 1) * group : 0;
}
__device__ __forceinline__ uint32_t tc_hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ bool tc_elect() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// 32 consecutive 32-bit columns of this thread's TMEM lane: the load, and the wait for every
// load so far (the registers hold nothing before it).
__device__ __forceinline__ void tc_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
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
__device__ __forceinline__ void tc_ld32_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
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

template <int D, bool F16>
__global__ void __launch_bounds__(kTcThreads, 1)
    lora_kv4_weights_tc_kernel(const __grid_constant__ TcParams p) {
  using B = Kv4Block<D>;
  constexpr int ATOMS = D / 64;                        // 128-byte atoms of a row
  constexpr uint32_t kAtom = 128 * 128;                // 128 rows of one
  constexpr uint32_t kTile = ATOMS * kAtom;            // an operand tile of 128 rows
  constexpr uint32_t kOffQ = 4 * kTile;                // behind two items' K
  constexpr uint32_t kOffShared = kOffQ + 2 * kTile;
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
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sh.q_full[i]), kTcRowThreads + (p.wait_fault ? 1 : 0));
      mbar_init(bar(sh.q_empty[i]), 1);
      mbar_init(bar(sh.k_full[i]), 4);
      mbar_init(bar(sh.k_empty[i]), 1);
      mbar_init(bar(sh.s_full[i]), 1);
      mbar_init(bar(sh.s_empty[i]), 8);
    }
    for (int i = 0; i < kTcAhead; ++i) mbar_init(bar(sh.l_full[i]), 3);
    mbar_init(bar(sh.drain), 1);
    fence_mbar_init();
    sh.abort = 0;
  }
  if (warp == 15) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     smem_u32(&sh.taddr)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  const CtaAbort cta_abort{&sh.abort, p.wait_limit_ns};
  pdl_wait();
  pdl_launch_dependents();

  // ---- the pairs of sequence and key tile, and their order
  const int per_thread = (a.num_seqs + kTcThreads - 1) / kTcThreads;
  long long mine = 0;
  for (int i = 0; i < per_thread; ++i) {
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
  if (lane == 31) sh.warp_long[warp] = run;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long before = 0, pairs = 0;
#pragma unroll
  for (int w = 0; w < kTcWarps; ++w) {
    if (w < warp) before += sh.warp_long[w];
    pairs += sh.warp_long[w];
  }
  before += run - mine;
  sh.prefix[tid] = before;
  const bool sorted = pairs <= kTcPairs;
  if (sorted && mine > 0) {
    int at = static_cast<int>(before);
    for (int i = 0; i < per_thread; ++i) {
      const int b = tid * per_thread + i;
      if (b >= a.num_seqs) break;
      const WeightSeq s = WeightSeq::of(a, b);
      if (!tc_mine(s, group, p.max_packed_rows)) continue;
      const int first = tc_first(s, a.window), n = tc_count(s, a.window);
      for (int k = 0; k < n; ++k, ++at) {
        int row0, rows;
        tc_rows(s, first + k, group, a.window, row0, rows);
        sh.pair_b[at] = b, sh.pair_kt[at] = first + k, sh.pair_tiles[at] = (rows + kTcRows - 1) / kTcRows;
      }
    }
  }
  __syncthreads();
  if (sorted && tid < pairs) {  // a pair's place: those of more tiles first, then in their own order
    const int n = sh.pair_tiles[tid];
    int place = 0;
    for (int i = 0; i < static_cast<int>(pairs); ++i) {
      const int m = sh.pair_tiles[i];
      place += m > n || (m == n && i < tid) ? 1 : 0;
    }
    sh.sorted[place] = tid;
  }
  __syncthreads();
  const uint32_t taddr = sh.taddr;
  const long long items = pairs * a.num_kv_heads;
  // The CTA's k-th item (by whole warps); false: there is none.
  auto item_at = [&](long long k, TcItem& it) -> bool {
    const long long G = gridDim.x, c = blockIdx.x;
    const long long e = k * G + ((k & 1) && sorted ? G - 1 - c : c);
    if (e >= items) return false;
    const long long pr = quotient(e, a.num_kv_heads);
    it.h = static_cast<int>(e - pr * a.num_kv_heads);
    if (sorted) {
      const int at = sh.sorted[pr];
      it.b = sh.pair_b[at], it.kt = sh.pair_kt[at];
      it.seq = WeightSeq::of(a, it.b);
    } else {
      const int lo = last_not_past<kTcWarps>(sh.prefix, pr, lane);
      long long off = pr - sh.prefix[lo];
      for (it.b = lo * per_thread;; ++it.b) {
        it.seq = WeightSeq::of(a, it.b);
        const int n = tc_mine(it.seq, group, p.max_packed_rows) ? tc_count(it.seq, a.window) : 0;
        if (off < n) break;
        off -= n;
      }
      it.kt = tc_first(it.seq, a.window) + static_cast<int>(off);
    }
    tc_rows(it.seq, it.kt, group, a.window, it.row0, it.rows);
    return true;
  };
  // (a place past the end in one round is followed by none that is not)
  auto given_up = [&]() { return __any_sync(0xffffffffu, cta_abort.raised()) != 0; };

  if (warp < 8) {
    // -------------------------------------------------------------- sums
    const int sub = warp >> 2, key_in = sub * 128 + (warp & 3) * 32 + lane;
    const uint32_t tS = taddr + (static_cast<uint32_t>((warp & 3) * 32) << 16) + sub * kTcRows;
    const float c = score_factor(1.0f, a.score_scale * kTcLog2e);
    uint32_t t = 0;  // row tiles so far
    bool lost = false;
    TcItem it;
    for (long long k = 0; item_at(k, it) && !given_up(); ++k) {
      const int j = it.kt * kTcKeys + key_in;
      const bool there = j < it.seq.end && j >= it.seq.first_key(0, a.window);
      const int before_rows = it.seq.kv - it.seq.rows;
      float* w = a.weights + (static_cast<long long>(it.b) * a.num_kv_heads + it.h) * a.capacity + j;
      float old = 0.0f;
      bool draws = false;
      if (there) {
        const int page = __ldg(a.page_table + it.b * a.table_stride + j / a.page_size);
        draws = page >= 0 && page < a.num_pages;
        lost = lost || !draws;
        if (j < before_rows) old = *w;
      }
      // the packed rows that see this key: [see0, see1)
      const int see0 = max(j - before_rows, 0) * group;
      int see1 = it.row0 + it.rows;
      if (a.window > 0) {
        const long long i1 = static_cast<long long>(j) + a.window - before_rows;  // behind the last
        if (i1 * group < see1) see1 = static_cast<int>(max(i1 * group, 0ll));
      }
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      const int tiles = it.tiles();
      for (int x = 0; x < tiles; ++x, ++t) {
        const int buf = t & 1, slot = t % kTcAhead;
        cta_abort.wait(bar(sh.l_full[slot]), (t / kTcAhead) & 1);
        cta_abort.wait(bar(sh.s_full[buf]), (t >> 1) & 1);
        __syncwarp();
        tc_fence_after();
        const int r0 = it.row0 + x * kTcRows;
        const int lo = max(see0 - r0, 0), hi = min(see1 - r0, kTcRows);  // columns that count
        const bool masked = __any_sync(0xffffffffu, lo > 0 || hi < kTcRows) || sh.odd[slot] != 0;
        const uint32_t at = tS + buf * 2 * kTcRows;
        const float* neg = sh.neg[slot];
        if (!masked) {
          uint32_t v[2][32];
          tc_ld32_start(at, v[0]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t (&s)[32] = v[q & 1];
            tc_ld32_wait(s);
            if (q < 3) tc_ld32_start(at + 32 * (q + 1), v[(q + 1) & 1]);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 n = *reinterpret_cast<const float4*>(neg + 32 * q + e);
              float x0, x1, x2, x3;
              tc_fma2(x0, x1, s[e], s[e + 1], c, n.x, n.y);
              tc_fma2(x2, x3, s[e + 2], s[e + 3], c, n.z, n.w);
              tc_add2(sum[0], sum[1], exp2_approx(x0), exp2_approx(x1));
              tc_add2(sum[2], sum[3], exp2_approx(x2), exp2_approx(x3));
            }
          }
        } else {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            if (!__any_sync(0xffffffffu, lo < 32 * q + 32 && hi > 32 * q)) continue;
            uint32_t s[32];
            tc_ld32_start(at + 32 * q, s);
            tc_ld32_wait(s);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float n = neg[32 * q + e];
              const float x0 = exp2_approx(fmaf(__uint_as_float(s[e]), c, n));
              const bool in = 32 * q + e >= lo && 32 * q + e < hi && n != -INFINITY;
              sum[e & 3] += in ? x0 : 0.0f;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !cta_abort.raised()) mbar_arrive(bar(sh.s_empty[buf]));
      }
      if (there && !cta_abort.raised())
        *w = old + (draws ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.0f);
    }
    if (lost && a.status) atomicOr(a.status, kStatusBadSlot);
  } else if (warp < 12) {
    // -------------------------------------------------------------- keys
    const int r = tid - 256;
    const int page_blocks = a.page_size / 16;
    uint4 codes[2][D / 32];
    uint32_t scales[2][D / 64];
    auto load = [&](const TcItem& it) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int j = it.kt * kTcKeys + s * 128 + r;
        const uint8_t* blk = nullptr;
        if (j < it.seq.end && j >= it.seq.first_key(0, a.window)) {
          const int pg = j / a.page_size, in = (j - pg * a.page_size) / 16;
          const int page = __ldg(a.page_table + it.b * a.table_stride + pg);
          if (page >= 0 && page < a.num_pages)
            blk = a.cache + ((static_cast<long long>(page) * a.num_kv_heads + it.h) * page_blocks + in) * B::kBytes;
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          codes[s][c] = blk ? __ldg(reinterpret_cast<const uint4*>(blk + (j & 15) * B::kCodeRow) + c)
                            : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          scales[s][c] = blk ? __ldg(reinterpret_cast<const uint32_t*>(blk + B::kKScale + (j & 15) * B::kScaleRow) + c)
                             : 0u;
      }
    };
    TcItem it;
    uint32_t n = 0;  // items with products so far
    bool more = item_at(0, it);
    if (more) load(it);
    for (long long k = 0; more && !given_up(); ++k) {
      const bool used = it.rows > 0;
      if (used) {
        const int st = n & 1;
        if (n >= 2) cta_abort.wait(bar(sh.k_empty[st]), ((n >> 1) - 1) & 1);
        __syncwarp();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          unsigned char* tile = smem + (st * 2 + s) * kTile;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {  // 32 dimensions: two scales, four 16-byte chunks
            const uint32_t h = e4m3x2_to_f16(scales[s][c / 2] >> (16 * (c & 1)));
            const uint32_t f[2] = {__byte_perm(h, h, 0x1010), __byte_perm(h, h, 0x3232)};
            const uint32_t x[4] = {codes[s][c].x, codes[s][c].y, codes[s][c].z, codes[s][c].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t v[4];
              e2m1x8_to_f16(x[e], v);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                v[i] = tc_hmul2(v[i], f[e / 2]);
                if constexpr (!F16) {
                  const float2 u = unpack_f16x2(v[i]);
                  v[i] = pack_bf16x2(u.x, u.y);
                }
              }
              const int ch = 4 * c + e;
              *reinterpret_cast<uint4*>(tile + (ch >> 3) * kAtom + swz128(r, ch & 7)) =
                  make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0 && !cta_abort.raised()) mbar_arrive(bar(sh.k_full[st]));
        ++n;
      }
      more = item_at(k + 1, it);
      if (more) load(it);
    }
  } else if (warp < 15) {
    // -------------------------------------------------------------- rows
    constexpr int CHUNKS = D / 8;  // 16-byte chunks of a row
    const int r = tid - 384;
    bool odd_path = false;
    uint32_t t = 0;
    TcItem it;
    for (long long k = 0; item_at(k, it) && !given_up(); ++k) {
      const int tiles = it.tiles();
      for (int x = 0; x < tiles; ++x, ++t) {
        const int st = t & 1, slot = t % kTcAhead;
        if (t >= 2) cta_abort.wait(bar(sh.q_empty[st]), ((t >> 1) - 1) & 1);
        __syncwarp();
        const int r0 = it.row0 + x * kTcRows, cols = min(it.row0 + it.rows - r0, kTcRows);
        const int padded = (cols + 15) & ~15;
        for (int u = r; u < padded * CHUNKS; u += kTcRowThreads) {
          const int c = u / CHUNKS, ch = u % CHUNKS, row = r0 + min(c, cols - 1);
          const int i = row / group, head = it.h * group + row - i * group;
          const int at = it.seq.row_in_q(a, it.b, i);
          const bool real = c < cols && at >= 0;
          cp_async_16(sbase + kOffQ + st * kTile + (ch >> 3) * kAtom + swz128(c, ch & 7),
                      a.q + (real ? at : 0) * a.q_stride + head * D + 8 * ch, real);
        }
        // (the copies arrive themselves as they land; the products' warp fences)
        if (!given_up()) cp_async_mbar_arrive(bar(sh.q_full[st]));
        bool odd = false;
        for (int c = r; c < kTcRows; c += kTcRowThreads) {
          float lse = -INFINITY;
          if (c < cols) {
            const int row = r0 + c, i = row / group, head = it.h * group + row - i * group;
            const int at = it.seq.row_in_q(a, it.b, i);
            if (at >= 0) lse = __ldg(a.lse + static_cast<long long>(at) * a.num_q_heads + head);
            else odd_path = true;
            odd = odd || lse == -INFINITY;
          }
          sh.neg[slot][c] = lse == -INFINITY ? -INFINITY : -(lse * kTcLog2e);
        }
        // (all three warps write the flag's word before any lane of another reads it: l_full)
        odd = __any_sync(0xffffffffu, odd);
        if (lane == 0) {
          reinterpret_cast<volatile unsigned char*>(&sh.odd[slot])[warp - 12] = odd ? 1 : 0;
          if (warp == 12) reinterpret_cast<volatile unsigned char*>(&sh.odd[slot])[3] = 0;
        }
        __syncwarp();
        if (lane == 0 && !cta_abort.raised()) mbar_arrive(bar(sh.l_full[slot]));
      }
    }
    if (odd_path && a.status) atomicOr(a.status, kStatusBadLength);
  } else {
    // -------------------------------------------------------------- products
    uint32_t t = 0, n = 0;
    TcItem it;
    bool ok = true;
    for (long long k = 0; ok && item_at(k, it); ++k) {
      const int tiles = it.tiles();
      if (tiles == 0) continue;
      const int ka = n & 1;
      ok = __all_sync(0xffffffffu, cta_abort.wait(bar(sh.k_full[ka]), (n >> 1) & 1));
      for (int x = 0; ok && x < tiles; ++x, ++t) {
        const int st = t & 1;
        ok = cta_abort.wait(bar(sh.q_full[st]), (t >> 1) & 1);
        if (t >= 2) ok = cta_abort.wait(bar(sh.s_empty[st]), ((t >> 1) - 1) & 1) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        fence_proxy_async();  // the rows were written by copies of other threads
        tc_fence_after();
        const int cols = min(it.rows - x * kTcRows, kTcRows);
        const uint32_t idesc = kIdesc | (static_cast<uint32_t>((cols + 15) >> 4) << 18);
        if (tc_elect()) {
          const uint64_t dq = umma_desc_sw128(sbase + kOffQ + st * kTile, 16, 1024);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint64_t dk = umma_desc_sw128(sbase + (ka * 2 + s) * kTile, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * kAtom + (kk & 3) * 32) >> 4;
              umma_f16(taddr + (st * 2 + s) * kTcRows, dk + off, dq + off, idesc, kk != 0 ? 1u : 0u);
            }
          }
          umma_commit(bar(sh.s_full[st]));
          umma_commit(bar(sh.q_empty[st]));
          if (x + 1 == tiles) umma_commit(bar(sh.k_empty[ka]));
        }
        __syncwarp();
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
  if (warp == 15)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(512u)
                 : "memory");
  if (tid == 0 && cta_abort.raised() && a.status) atomicOr(a.status, kStatusTimeout);
}

int launch_kv4_weights_tc(const Kv4WeightsArgs& a, int max_packed_rows, bool f16, cudaStream_t stream) {
  const void* fn =
      a.head_dim == 64 ? (f16 ? reinterpret_cast<const void*>(lora_kv4_weights_tc_kernel<64, true>)
                              : reinterpret_cast<const void*>(lora_kv4_weights_tc_kernel<64, false>))
                       : (f16 ? reinterpret_cast<const void*>(lora_kv4_weights_tc_kernel<128, true>)
                              : reinterpret_cast<const void*>(lora_kv4_weights_tc_kernel<128, false>));
  const size_t smem = 1024 + 6 * static_cast<size_t>(a.head_dim / 64) * 128 * 128 + sizeof(TcShared);
  if (ensure_smem_attr(fn, smem) != 0) return -6;
  const int sms = device_sm_count();
  if (sms <= 0) return -6;
  TcParams p;
  p.a = a;
  p.max_packed_rows = max_packed_rows;
  p.wait_fault = wait_fault() ? 1 : 0;
  p.wait_limit_ns = p.wait_fault ? kTestWaitLimitNs : kWaitLimitNs;
  return launch_pdl(fn, dim3(sms), dim3(kTcThreads), smem, stream, 0, &p);
}

}  // namespace grg
