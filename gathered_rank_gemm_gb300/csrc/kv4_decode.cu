// Attention over the 4-bit paged cache for sequences with few query rows
// (decode, drafted tokens): rows x heads of one key head are packed into groups of
// 8 * NT rows, and one pass over the group's keys forms the scores, the running
// softmax and the weighted sum of the values.
//
// Mathematics, for a block of 16 keys (mma.sync m16n8k16, fp16 operands, fp32
// accumulators; the codes times their e4m3 scales are exact in fp16):
//   S[16 keys x 8 rows] = K Q^T, the keys as M, so a group of 8 rows wastes
//   nothing;  p = 2^(S c - m), m the running maximum in units of log2;
//   O[16 dims x 8 rows] += V^T P, the P fragments turned by movmatrix.
// A warp holds the rows' O and the maximum and sum per row in registers; keys
// come two blocks at a time through a ring of bulk copies in shared memory, one
// copy per block (a block's codes and scales lie together).  The maximum is
// moved only when a block exceeds it by 2^6 or more: p stays below 2^6, far
// inside fp16, and the rescaling of O almost never runs.
//
// Work: the blocks of all (sequence, row group, key head) items in one line,
// cut into equal runs whatever the lengths, so one long sequence fills the GPU
// as well as many short ones.  A run goes to a warp, or, where an item would
// span more than 16 warps' runs, to a whole CTA whose warps share its blocks
// and join in shared memory.  Items that were cut leave (m, l, O) partials in
// the workspace; the last of an item's runs to finish joins them, always in
// run order, so results do not depend on timing.
#include "kv4_attention.cuh"
#include "kv4_attention.h"
#include "launch.h"

namespace grg {

namespace {
constexpr int kDecThreads = 256;
constexpr int kDecWarps = kDecThreads / 32;
constexpr int kDecCtasMax = 2 * 160;  // CTAs that the workspace has room for
constexpr int kPartialSlots = kDecCtasMax * kDecWarps * 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct DecodeParams {
  Kv4AttnArgs a;
  uint32_t* counters;  // [kDecCtasMax * kDecWarps], zero between calls
  float* part_o;       // [slot][8 * NT][D]
  float2* part_ml;     // [slot][8 * NT]
  int max_packed_rows; // sequences with more packed rows are not this kernel's
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
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(a));
  return r;
}
}  // namespace

// One item: a group of packed rows of a sequence and a key head, and its keys.
struct DecItem {
  int blk0;  // first block of 16 keys
  int nb;    // blocks (1 where no row sees a key: nothing is loaded then)
  int hi;    // keys [.., hi) are seen by some row; 0: none
};
template <int ROWS>
__device__ __forceinline__ DecItem dec_item(const Kv4Seq& s, int group, int rg, int window) {
  const int i0 = rg * ROWS / group, i1 = (min(s.take * group, (rg + 1) * ROWS) - 1) / group;
  const int hi = s.pos(i1) + 1, lo = s.first_key(i0, window);
  DecItem it;
  it.blk0 = lo / 16;
  it.hi = hi > lo ? hi : 0;
  it.nb = hi > lo ? (hi + 15) / 16 - it.blk0 : 1;
  return it;
}

template <int D, int NT, bool F16>
__global__ void __launch_bounds__(kDecThreads, NT == 1 ? 2 : 1)
    lora_kv4_decode_kernel(const __grid_constant__ DecodeParams p) {
  using B = Kv4Block<D>;
  constexpr int ROWS = 8 * NT;
  constexpr int KS = D / 16;              // k steps of S, and 16-dimension tiles of O
  constexpr int STAGES = NT == 1 ? 3 : 4; // pairs of blocks in a warp's ring
  constexpr int kStage = 2 * B::kBytes;
  constexpr int kRing = STAGES * kStage;
  constexpr int PITCH = D + 4;            // floats of a row's partial in shared memory
  static_assert(kRing >= ROWS * PITCH * 4, "a warp's partial fits its ring");

  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t s_bar[kDecWarps * STAGES];
  __shared__ long long s_prefix[kDecThreads + 1];
  __shared__ long long s_warp[2][kDecWarps];
  __shared__ int s_abort, s_last;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const Kv4AttnArgs& a = p.a;
  const int group = a.num_q_heads / a.num_kv_heads;
  const uint32_t bars = smem_u32(s_bar + warp * STAGES);
  if (lane == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(bars + 8 * i, 1 + (p.wait_fault ? 1 : 0));
    fence_mbar_init();
  }
  if (tid == 0) s_abort = 0;
  const CtaAbort cta_abort{&s_abort, p.wait_limit_ns};
  pdl_wait();
  pdl_launch_dependents();

  // ---- the line of units (blocks), by sequence: a prefix sum over the threads'
  // runs of sequences
  const int per_thread = (a.num_seqs + kDecThreads - 1) / kDecThreads;
  auto units_of = [&](int b, int& items) -> long long {
    const Kv4Seq s = Kv4Seq::of(a, b);
    items = 0;
    if (s.odd && blockIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadLength);
    if (s.take == 0 || static_cast<long long>(s.take) * group > p.max_packed_rows) return 0;
    const int ng = (s.take * group + ROWS - 1) / ROWS;
    long long n = 0;
    for (int rg = 0; rg < ng; ++rg) n += dec_item<ROWS>(s, group, rg, a.window).nb;
    items = ng * a.num_kv_heads;
    return n * a.num_kv_heads;
  };
  long long mine = 0, my_items = 0;
  for (int i = 0; i < per_thread; ++i) {
    const int b = tid * per_thread + i;
    if (b < a.num_seqs) {
      int items;
      mine += units_of(b, items);
      my_items += items;
    }
  }
  long long run = mine, all_items = my_items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += v;
    all_items += __shfl_xor_sync(0xffffffffu, all_items, o);
  }
  if (lane == 31) s_warp[0][warp] = run;
  if (lane == 0) s_warp[1][warp] = all_items;
  __syncthreads();
  long long before = 0, total = 0, items = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) before += s_warp[0][w];
    total += s_warp[0][w];
    items += s_warp[1][w];
  }
  s_prefix[tid] = before + run - mine;
  if (tid == 0) s_prefix[kDecThreads] = total;
  __syncthreads();
  if (total == 0) return;

  // ---- runs of warps or of CTAs
  const long long warps_all = static_cast<long long>(gridDim.x) * kDecWarps;
  const long long per_warp = max((total + warps_all - 1) / warps_all, 2ll);
  const bool team = total > 16 * per_warp * items;  // an item would span over 16 warps' runs
  const long long per = team ? max((total + gridDim.x - 1) / gridDim.x, 2ll * kDecWarps) : per_warp;
  const int worker = team ? blockIdx.x : blockIdx.x * kDecWarps + warp;
  const int TW = team ? kDecWarps : 1, wt = team ? warp : 0;
  auto team_sync = [&]() {
    if (team) __syncthreads(); else __syncwarp();
  };
  unsigned char* ring = smem + warp * kRing;
  const uint32_t ring_u = smem_u32(ring);
  float* own = reinterpret_cast<float*>(ring);  // the warp's partial, once its ring is idle
  uint32_t fills = 0;                           // copies awaited so far (stage and phase)

  long long u = worker * per;
  const long long u_end = min(u + per, total);
  if (u >= u_end) return;  // a whole team or a lone warp
  // the sequence, row group, key head and offset of unit u
  int b = 0, rg = 0, h = 0;
  long long off = 0;
  {
    int lo = 0, hi = kDecThreads;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (s_prefix[mid] <= u) lo = mid; else hi = mid;
    }
    off = u - s_prefix[lo];
    b = lo * per_thread;
    int ignored;
    for (long long n; off >= (n = units_of(b, ignored)); ++b) off -= n;
  }
  Kv4Seq seq = Kv4Seq::of(a, b);
  DecItem item = dec_item<ROWS>(seq, group, 0, a.window);
  while (off >= static_cast<long long>(item.nb) * a.num_kv_heads) {
    off -= static_cast<long long>(item.nb) * a.num_kv_heads;
    item = dec_item<ROWS>(seq, group, ++rg, a.window);
  }
  h = static_cast<int>(off / item.nb);
  int o = static_cast<int>(off % item.nb);

  while (true) {
    const int take = static_cast<int>(min(static_cast<long long>(item.nb - o), u_end - u));
    const int first_blk = item.blk0 + o;
    const int packed = seq.take * group;  // packed rows of the sequence
    const int row0 = rg * ROWS;
    const int live_rows = min(packed - row0, ROWS);

    // ---- the rows' queries as B fragments, in fp16, and what undoes their factor
    uint32_t qf[NT][KS][2];
    float cf[NT][2];
    int pos[NT][2], lo[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + g;
      float v[KS * 4], top = 0.0f;
#pragma unroll
      for (int i = 0; i < KS * 4; ++i) v[i] = 0.0f;
      if (r < packed) {
        const uint16_t* src = a.q + (seq.q0 + r / group) * a.q_stride + (h * group + r % group) * D +
                              t4 * (D / 4);
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(src) + i);
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = unpack_t<F16>(x[k]);
            v[8 * i + 2 * k] = f.x, v[8 * i + 2 * k + 1] = f.y;
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
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
        cf[nt][c] = __shfl_sync(0xffffffffu, down, (2 * t4 + c) * 4) * (a.score_scale * kLog2e);
        const int rr = min(row0 + nt * 8 + 2 * t4 + c, packed - 1) / group;
        pos[nt][c] = seq.pos(rr);
        lo[nt][c] = seq.first_key(rr, a.window);
      }
    }
    const int pos_min = seq.pos(row0 / group), pos_max = item.hi - 1;
    const int lo_max = seq.first_key((row0 + live_rows - 1) / group, a.window);

    float acc[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) m[nt][c] = -INFINITY, l[nt][c] = 0.0f;
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[nt][i][c] = 0.0f;
    }
    bool poison = false;  // a NaN scale of V among keys that some rows must not see

    // ---- this warp's pairs of blocks: pair k covers blocks 2 q, 2 q + 1 of the run, q = wt + TW k
    const int pairs = (take + 1) / 2;
    const int np = item.hi > 0 && !p.wait_fault ? (pairs - wt + TW - 1) / TW : (p.wait_fault ? 1 : 0);
    const int32_t* table = a.page_table + static_cast<long long>(b) * a.table_stride;
    const int page_blocks = a.page_size / 16;
    // block addresses: 16 pairs at a time, lane l holds block l & 1 of pair l / 2 (null: not there)
    auto address = [&](int k0) -> const unsigned char* {
      const int q = wt + TW * (k0 + (lane >> 1));
      const int i = 2 * q + (lane & 1);
      if (i >= take) return nullptr;
      const int blk = first_blk + i, pg = blk / page_blocks;
      const int page = __ldg(table + pg);
      if (page < 0 || page >= a.num_pages) {
        if (a.status) atomicOr(a.status, kStatusBadSlot);
        return nullptr;
      }
      return a.cache + ((static_cast<long long>(page) * a.num_kv_heads + h) * page_blocks +
                        (blk - pg * page_blocks)) * B::kBytes;
    };
    const unsigned char* now = np > 0 ? address(0) : nullptr;
    uint32_t there = 0;  // two bits per stage: which blocks of the pair exist
    auto issue = [&](int k) {
      if ((k & 15) == 0 && k > 0) now = address(k);
      const unsigned long long at = reinterpret_cast<unsigned long long>(now);
      const unsigned long long x0 = __shfl_sync(0xffffffffu, at, 2 * (k & 15));
      const unsigned long long x1 = __shfl_sync(0xffffffffu, at, 2 * (k & 15) + 1);
      const int s = (fills + k) % STAGES;
      there = (there & ~(3u << (2 * s))) | (((x0 ? 1u : 0u) | (x1 ? 2u : 0u)) << (2 * s));
      if (lane == 0 && !cta_abort.raised()) {
        const uint32_t bar = bars + 8 * s, dst = ring_u + s * kStage;
        const uint32_t bytes = ((x0 ? 1 : 0) + (x1 ? 1 : 0)) * B::kBytes;
        mbar_arrive_expect_tx(bar, p.wait_fault ? 0 : bytes);
        if (!p.wait_fault) {
          if (x0) bulk_g2s(dst, reinterpret_cast<const void*>(x0), B::kBytes, bar);
          if (x1) bulk_g2s(dst + B::kBytes, reinterpret_cast<const void*>(x1), B::kBytes, bar);
        }
      }
    };
    int issued = 0;
    for (; issued < min(np, STAGES); ++issued) issue(issued);

    int k = 0;
    for (; k < np; ++k) {
      const int s = (fills + k) % STAGES;
      if (!__all_sync(0xffffffffu, cta_abort.wait(bars + 8 * s, ((fills + k) / STAGES) & 1))) break;
      const unsigned char* stage = ring + s * kStage;
      const int tok = 16 * (first_blk + 2 * (wt + TW * k));  // the pair's first key
      const uint32_t have = (there >> (2 * s)) & 3u;
      const bool masked = tok + 31 > pos_min || tok < lo_max || have != 3u;
      // key of this thread's S rows g and g + 8 (parities alternate: no bank conflicts)
      const int kr = g ^ ((g >> 1) & 1);

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
          sa[0] = prmt(ha, ha, 0x1010), sa[1] = prmt(ha, ha, 0x3232);
          sb[0] = prmt(hb, hb, 0x1010), sb[1] = prmt(hb, hb, 0x3232);
        } else {
          const uint2 va = *reinterpret_cast<const uint2*>(blk + kr * 32 + 8 * t4);
          const uint2 vb = *reinterpret_cast<const uint2*>(blk + (kr + 8) * 32 + 8 * t4);
          ca[0] = va.x, ca[1] = va.y, cb[0] = vb.x, cb[1] = vb.y;
          const uint32_t ha = e4m3x2_to_f16(blk[B::kKScale + kr * 4 + t4]);
          const uint32_t hb = e4m3x2_to_f16(blk[B::kKScale + (kr + 8) * 4 + t4]);
          sa[0] = sa[1] = prmt(ha, ha, 0x1010);
          sb[0] = sb[1] = prmt(hb, hb, 0x1010);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[nt][x][c] = 0.0f;
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
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(sc[nt][x], frag, qf[nt][2 * w + j][0], qf[nt][2 * w + j][1]);
          }
        }
      }

      // ---- running maximum (rarely moved) and the probabilities
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
          float v = fmaxf(fmaxf(sc[nt][0][c], sc[nt][0][c + 2]), fmaxf(sc[nt][1][c], sc[nt][1][c + 2]));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          mx[nt][c] = v * cf[nt][c];
          move = move || mx[nt][c] > m[nt][c] + 6.0f;
        }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float to = fmaxf(m[nt][c], mx[nt][c]);
            const float f = m[nt][c] == -INFINITY ? 0.0f : exp2_approx(m[nt][c] - to);
            m[nt][c] = to;
            l[nt][c] *= f;
#pragma unroll
            for (int i = 0; i < KS; ++i) acc[nt][i][c] *= f, acc[nt][i][c + 2] *= f;
          }
      }
      uint32_t pb[NT][2][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float m0 = m[nt][0] == -INFINITY ? 0.0f : m[nt][0];
        const float m1 = m[nt][1] == -INFINITY ? 0.0f : m[nt][1];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float p0 = exp2_approx(fmaf(sc[nt][x][0], cf[nt][0], -m0));
          const float p1 = exp2_approx(fmaf(sc[nt][x][1], cf[nt][1], -m1));
          const float p2 = exp2_approx(fmaf(sc[nt][x][2], cf[nt][0], -m0));
          const float p3 = exp2_approx(fmaf(sc[nt][x][3], cf[nt][1], -m1));
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
        const uint32_t s01 = e4m3x2_to_f16(e0 | (e1 << 8)), s23 = e4m3x2_to_f16(e2 | (e3 << 8));
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
              mma_f16(acc[nt][4 * w + i], frag, pb[nt][x][0], pb[nt][x][1]);
          }
        }
      }
      __syncwarp();
      if (issued < np) issue(issued++);
    }
    if (k < np)  // gave up: what is still on its way lands before the ring is left
      for (; k < issued && !p.wait_fault; ++k)
        mbar_drain(bars + 8 * ((fills + k) % STAGES), ((fills + k) / STAGES) & 1, p.wait_limit_ns);
    fills += np;

    // ---- join: sums over the lanes that share a row
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 4);
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 8);
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 16);
      }
    if (__any_sync(0xffffffffu, poison)) {
      // rare: which of its 16 dimensions' scales are NaN at keys a row sees
      for (int i = 0; i < 2 * pairs; ++i) {
        if (TW > 1 && (i / 2) % TW != wt) continue;
        const int blk = first_blk + i, pg = blk / page_blocks;
        if (i >= take || blk * 16 >= item.hi) continue;
        const int page = __ldg(table + pg);
        if (page < 0 || page >= a.num_pages) continue;
        const unsigned char* at =
            a.cache + ((static_cast<long long>(page) * a.num_kv_heads + h) * page_blocks +
                       (blk - pg * page_blocks)) * B::kBytes + B::kVScale + (D == 128 ? g : g / 2);
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

    // The joined rows in the team's shared memory: [row][D], then (m, l) at D.
    auto put = [&](float* dst) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = nt * 8 + 2 * t4 + c;
          if (r >= live_rows) continue;
          float* row = dst + r * PITCH;
#pragma unroll
          for (int i = 0; i < KS; ++i)
            *reinterpret_cast<float2*>(row + (D / 8) * g + 2 * i) =
                make_float2(acc[nt][i][c], acc[nt][i][c + 2]);
          if (g == 0) *reinterpret_cast<float2*>(row + D) = make_float2(m[nt][c], l[nt][c]);
        }
    };
    // Joins the team's warps' rows and hands each (row, 4 dimensions) on.
    auto join = [&](auto&& sink) {
      const int step = TW * 32;
      for (int i = wt * 32 + lane; i < live_rows * (D / 4); i += step) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        const float* base = reinterpret_cast<const float*>(smem + (team ? 0 : warp) * kRing) + r * PITCH;
        float top = -INFINITY;
        for (int w = 0; w < TW; ++w)
          top = fmaxf(top, base[static_cast<size_t>(w) * (kRing / 4) + D]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.0f;
        for (int w = 0; w < TW; ++w) {
          const float* part = base + static_cast<size_t>(w) * (kRing / 4);
          const float2 ml = *reinterpret_cast<const float2*>(part + D);
          const float f = ml.x == -INFINITY ? 0.0f : exp2_approx(ml.x - top);
          const float4 x = *reinterpret_cast<const float4*>(part + d);
          // a part without keys adds nothing (its sums are zero, or NaN from NaN scores)
          sum += ml.x == -INFINITY ? ml.y : ml.y * f;
          v.x += ml.x == -INFINITY ? x.x : x.x * f;
          v.y += ml.x == -INFINITY ? x.y : x.y * f;
          v.z += ml.x == -INFINITY ? x.z : x.z * f;
          v.w += ml.x == -INFINITY ? x.w : x.w * f;
        }
        sink(r, d, v, top, sum);
      }
    };
    auto to_output = [&](int r, int d, float4 v, float top, float sum) {
      if (cta_abort.raised()) return;
      const int pr = row0 + r, t = seq.q0 + pr / group, head = h * group + pr % group;
      const float inv = sum == 0.0f ? 0.0f : a.v_scale / sum;
      uint2 w;
      w.x = pack_t<F16>(v.x * inv, v.y * inv);
      w.y = pack_t<F16>(v.z * inv, v.w * inv);
      *reinterpret_cast<uint2*>(a.out + t * a.out_stride + head * D + d) = w;
      if (d == 0 && a.lse)
        a.lse[static_cast<long long>(t) * a.num_q_heads + head] =
            sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    };
    put(own);
    team_sync();
    if (take == item.nb) {
      join(to_output);
    } else {
      const long long start = u - o;
      const int w0 = static_cast<int>(start / per), w1 = static_cast<int>((start + item.nb - 1) / per);
      const long long slot = static_cast<long long>(worker) * 2 + (o == 0 ? 1 : 0);
      join([&](int r, int d, float4 v, float top, float sum) {
        *reinterpret_cast<float4*>(p.part_o + (slot * ROWS + r) * D + d) = v;
        if (d == 0) p.part_ml[slot * ROWS + r] = make_float2(top, sum);
      });
      __threadfence();
      team_sync();
      int last = 0;
      if (wt == 0 && lane == 0) {
        last = atomicAdd(p.counters + w0, 1u) == static_cast<uint32_t>(w1 - w0);
        if (last) p.counters[w0] = 0;
        __threadfence();
        if (team) s_last = last;
      }
      if (team) {
        __syncthreads();
        last = s_last;
      } else {
        last = __shfl_sync(0xffffffffu, last, 0);
      }
      if (last) {
        // every run of the item is there: each warp sums its share of them, in run order
        const int n = w1 - w0 + 1;
        for (int r = 0; r < live_rows; ++r) {
          float top = -INFINITY;
          for (int i = wt + TW * lane; i < n; i += TW * 32)
            top = fmaxf(top, __ldcg(&p.part_ml[((static_cast<long long>(w0) + i) * 2 + (i == 0)) * ROWS + r]).x);
#pragma unroll
          for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
          float v[D / 32] = {}, sum = 0.0f;
#pragma unroll 4
          for (int i = wt; i < n; i += TW) {
            const long long at = ((static_cast<long long>(w0) + i) * 2 + (i == 0)) * ROWS + r;
            const float2 ml = __ldcg(&p.part_ml[at]);
            const float f = ml.x == -INFINITY ? 1.0f : exp2_approx(ml.x - top);
            sum += ml.y * f;
            const float* src = p.part_o + at * D + lane * (D / 32);
#pragma unroll
            for (int e = 0; e < D / 32; e += 2) {
              const float2 x = __ldcg(reinterpret_cast<const float2*>(src + e));
              v[e] += x.x * f;
              v[e + 1] += x.y * f;
            }
          }
          float* row = own + r * PITCH;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) row[lane * (D / 32) + e] = v[e];
          if (lane == 0) *reinterpret_cast<float2*>(row + D) = make_float2(top, sum);
        }
        team_sync();
        join(to_output);
      }
    }
    fence_proxy_async();  // the rings' next writes are bulk copies
    team_sync();

    u += take;
    if (u >= u_end) break;
    o = 0;
    if (++h == a.num_kv_heads) {
      h = 0;
      ++rg;
      while (rg * ROWS >= seq.take * group) {  // the next sequence with rows of this kernel's
        rg = 0;
        do seq = Kv4Seq::of(a, ++b);
        while (static_cast<long long>(seq.take) * group > p.max_packed_rows);
      }
      item = dec_item<ROWS>(seq, group, rg, a.window);
    }
  }
  if (lane == 0 && cta_abort.raised() && a.status) atomicOr(a.status, kStatusTimeout);
}

namespace {
template <int D, int NT, bool F16>
int run_decode(const DecodeParams& q, cudaStream_t stream) {
  DecodeParams p = q;
  constexpr int stages = NT == 1 ? 3 : 4;
  const void* fn = reinterpret_cast<const void*>(lora_kv4_decode_kernel<D, NT, F16>);
  const size_t smem = static_cast<size_t>(kDecWarps) * stages * 2 * Kv4Block<D>::kBytes;
  if (ensure_smem_attr(fn, smem) != 0) return -6;
  const int sms = device_sm_count();
  if (sms <= 0) return -6;
  const int grid = min((NT == 1 ? 2 : 1) * sms, kDecCtasMax);
  return launch_pdl(fn, dim3(grid), dim3(kDecThreads), smem, stream, 0, &p);
}
constexpr size_t kCounterBytes = kDecCtasMax * kDecWarps * 4;
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
  p.wait_fault = wait_fault() ? 1 : 0;
  p.wait_limit_ns = p.wait_fault ? kTestWaitLimitNs : kWaitLimitNs;
  if (a.head_dim == 64)
    return wide ? (f16 ? run_decode<64, 2, true>(p, stream) : run_decode<64, 2, false>(p, stream))
                : (f16 ? run_decode<64, 1, true>(p, stream) : run_decode<64, 1, false>(p, stream));
  return wide ? (f16 ? run_decode<128, 2, true>(p, stream) : run_decode<128, 2, false>(p, stream))
              : (f16 ? run_decode<128, 1, true>(p, stream) : run_decode<128, 1, false>(p, stream));
}

}  // namespace grg
