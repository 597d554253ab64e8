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
// Warp roles (13 warps, one CTA per SM, persistent):
//  - warps 0-3 and 4-7, softmax of tile 0 and 1: a thread owns a row.  It writes
//    the row's q (scaled by a power of two into fp16's range) to shared memory,
//    then per key tile reads S, forms p with the running maximum (moved, and O
//    rescaled, only when a row's scores exceed it by 2^6 or more, which almost never
//    happens after the first tile) and stores P; at the end it writes the row of O.
//  - warps 8-11, keys and values: a thread owns a key of the tile.  It loads
//    the key's codes and scales into registers a tile ahead, and writes the fp16
//    values into the swizzled operand tiles (two stages each for K and V).
//  - warp 12 issues the products: while tile 0's softmax runs, tile 1's products
//    do, and the other way round.
// Work: the key tiles of all items in one line, cut into equal runs, one per CTA;
// an item that was cut leaves (m, l, O) partials, joined in run order by the last
// of its CTAs to finish (as in kv4_decode.cu).
#include "kv4_attention.cuh"
#include "kv4_attention.h"
#include "launch.h"

namespace grg {

namespace {
constexpr int kPreThreads = 13 * 32;
constexpr int kPreCtasMax = 160;  // CTAs that the workspace has room for
constexpr int kPreRows = 256;     // packed rows of an item
constexpr int kPreKeys = 128;     // keys of a tile
constexpr float kPreLog2e = 1.4426950408889634f;
constexpr float kPreLn2 = 0.6931471805599453f;

struct PrefillParams {
  Kv4AttnArgs a;
  uint32_t* counters;   // [kPreCtasMax], zero between calls
  float* part_o;        // [2 * kPreCtasMax][256][D]
  float2* part_ml;      // [2 * kPreCtasMax][256]
  int max_packed_rows;  // sequences with no more packed rows are not this kernel's
  unsigned long long wait_limit_ns;
  int wait_fault;
};

// Shared memory behind the operand tiles.
struct PreShared {
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t drain;
  // keys of a tile that exist; four tiles deep: a tile's words are rewritten only
  // after both softmaxes have taken the tile two further on
  uint32_t valid[4][4];
  uint32_t taddr;
  int abort, poison, last;
  long long prefix[kPreThreads + 1];
  long long warp_sum[13];
};

__device__ __forceinline__ uint32_t pre_hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
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
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void pre_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// An item's key tiles: [kt0, kt0 + nt); hi = 0 where no row sees a key.
struct PreItem {
  int kt0, nt, hi;
};
__device__ __forceinline__ PreItem pre_item(const Kv4Seq& s, int group, int rt, int window) {
  const int i0 = rt * kPreRows / group;
  const int i1 = (static_cast<int>(min(static_cast<long long>(s.take) * group,
                                       static_cast<long long>(rt + 1) * kPreRows)) - 1) / group;
  const int hi = s.pos(i1) + 1, lo = s.first_key(i0, window);
  PreItem it;
  it.kt0 = lo / kPreKeys;
  it.hi = hi > lo ? hi : 0;
  it.nt = hi > lo ? (hi + kPreKeys - 1) / kPreKeys - it.kt0 : 1;
  return it;
}
}  // namespace

template <int D, bool F16>
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

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Kv4AttnArgs& a = p.a;
  const int group = a.num_q_heads / a.num_kv_heads;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.q_full[i]), 128 + (p.wait_fault ? 1 : 0));
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.p_full[i]), 128);
      mbar_init(smem_u32(&sh.o_full[i]), 1);
      mbar_init(smem_u32(&sh.k_full[i]), 128);
      mbar_init(smem_u32(&sh.k_empty[i]), 1);
      mbar_init(smem_u32(&sh.v_full[i]), 128);
      mbar_init(smem_u32(&sh.v_empty[i]), 1);
    }
    mbar_init(smem_u32(&sh.drain), 1);
    fence_mbar_init();
    sh.abort = 0;
    sh.poison = 0;
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     smem_u32(&sh.taddr)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  const CtaAbort cta_abort{&sh.abort, p.wait_limit_ns};
  pdl_wait();
  pdl_launch_dependents();

  // ---- the line of units (key tiles): a prefix sum over the threads' runs of sequences
  const int per_thread = (a.num_seqs + kPreThreads - 1) / kPreThreads;
  auto mine_of = [&](const Kv4Seq& s) {
    return static_cast<long long>(s.take) * group > p.max_packed_rows;
  };
  auto tiles_of = [&](const Kv4Seq& s) {
    return static_cast<int>((static_cast<long long>(s.take) * group + kPreRows - 1) / kPreRows);
  };
  auto head_units = [&](const Kv4Seq& s) -> long long {  // units of one key head
    long long n = 0;
    if (mine_of(s)) {
      const int nr = tiles_of(s);
      for (int rt = 0; rt < nr; ++rt) n += pre_item(s, group, rt, a.window).nt;
    }
    return n;
  };
  long long mine = 0;
  for (int i = 0; i < per_thread; ++i) {
    const int b = tid * per_thread + i;
    if (b < a.num_seqs) mine += head_units(Kv4Seq::of(a, b)) * a.num_kv_heads;
  }
  long long run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += v;
  }
  if (lane == 31) sh.warp_sum[warp] = run;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < 13; ++w) {
    if (w < warp) before += sh.warp_sum[w];
    total += sh.warp_sum[w];
  }
  sh.prefix[tid] = before + run - mine;
  if (tid == 0) sh.prefix[kPreThreads] = total;
  __syncthreads();
  const uint32_t taddr = sh.taddr;

  const long long per = max((total + gridDim.x - 1) / static_cast<long long>(gridDim.x), 1ll);
  const long long u0 = blockIdx.x * per, u_end = min(u0 + per, total);

  // The CTA's parts of items, in order; every role walks the same list.
  struct Part {
    Kv4Seq seq;
    PreItem item;
    int b, h, rt;
    int o, take;  // key tiles [o, o + take) of the item
    long long u;  // first unit
  };
  auto set_part = [&](Part& q) {
    q.item = pre_item(q.seq, group, q.rt, a.window);
    q.take = static_cast<int>(min(static_cast<long long>(q.item.nt - q.o), u_end - q.u));
  };
  auto first_part = [&](Part& q) {
    int lo = 0, hi = kPreThreads;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (sh.prefix[mid] <= u0) lo = mid; else hi = mid;
    }
    long long off = u0 - sh.prefix[lo], n;
    q.b = lo * per_thread;
    while (true) {
      q.seq = Kv4Seq::of(a, q.b);
      n = head_units(q.seq);
      if (off < n * a.num_kv_heads) break;
      off -= n * a.num_kv_heads;
      ++q.b;
    }
    q.h = static_cast<int>(off / n);
    off -= q.h * n;
    q.rt = 0;
    while (true) {
      const int nt = pre_item(q.seq, group, q.rt, a.window).nt;
      if (off < nt) break;
      off -= nt;
      ++q.rt;
    }
    q.o = static_cast<int>(off);
    q.u = u0;
    set_part(q);
  };
  auto next_part = [&](Part& q) -> bool {
    q.u += q.take;
    if (q.u >= u_end) return false;
    q.o = 0;
    if (++q.rt == tiles_of(q.seq)) {
      q.rt = 0;
      if (++q.h == a.num_kv_heads) {
        q.h = 0;
        do q.seq = Kv4Seq::of(a, ++q.b);
        while (!mine_of(q.seq));
      }
    }
    set_part(q);
    return true;
  };
  auto live_rows = [&](const Part& q) {
    return static_cast<int>(min(static_cast<long long>(q.seq.take) * group - static_cast<long long>(q.rt) * kPreRows,
                                static_cast<long long>(kPreRows)));
  };
  auto bar = [&](uint64_t& b) { return smem_u32(&b); };

  if (u0 < u_end) {
    Part q;
    first_part(q);
    if (warp < 8) {
      // -------------------------------------------------------------- softmax
      const int t = warp >> 2;                    // tile
      const int row = (warp & 3) * 32 + lane;     // row of the tile, and TMEM lane
      const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t tS = taddr + lane_base + kColS + t * kPreKeys;
      const uint32_t tO = taddr + lane_base + kColO + t * D;
      uint32_t ns = 0, no = 0;  // S tiles and second products so far
      int stage_it = 0;         // key tiles so far (the stage's valid bits)
      do {
        const int live = live_rows(q);
        const int nact = live > 128 ? 2 : 1;
        if (t < nact) {
          const int packed0 = q.rt * kPreRows;
          const int pr = packed0 + min(t * 128 + row, live - 1);  // rows past the end repeat the last
          const int i = pr / group, head = q.h * group + pr % group, tok = q.seq.q0 + i;
          const int pos = q.seq.pos(i), lo = q.seq.first_key(i, a.window);
          // ---- the row of q, in fp16
          float down;
          {
            const uint16_t* src = a.q + tok * a.q_stride + head * D;
            uint4 w[D / 8];
            float top = 0.0f;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              w[c] = __ldg(reinterpret_cast<const uint4*>(src) + c);
              const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = unpack_t<F16>(x[e]);
                top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
              }
            }
            float up;
            row_factor(top, up, down);
            unsigned char* tile = smem + t * kTile;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = unpack_t<F16>(x[e]);
                y[e] = pack_f16x2(f.x * up, f.y * up);
              }
              *reinterpret_cast<uint4*>(tile + (c >> 3) * kAtom + swz128(row, c & 7)) =
                  make_uint4(y[0], y[1], y[2], y[3]);
            }
            fence_proxy_async();
            mbar_arrive(bar(sh.q_full[t]));
          }
          const float cf = down * (a.score_scale * kPreLog2e);
          float m = -INFINITY, l = 0.0f;
          for (int j = 0; j < q.take; ++j) {
            const int key0 = (q.item.kt0 + q.o + j) * kPreKeys;
            cta_abort.wait(bar(sh.s_full[t]), ns & 1);
            ++ns;
            __syncwarp();
            tc_fence_after();
            // keys of the tile that this row sees
            uint32_t seen[4];
            {
              const int hi_j = pos - key0, lo_j = lo - key0;
              const volatile uint32_t* valid = sh.valid[(stage_it + j) & 3];
              bool all = true;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int h = hi_j - 32 * c, g = lo_j - 32 * c;
                uint32_t s = valid[c];
                if (h < 31) s &= h < 0 ? 0u : (2u << h) - 1u;
                if (g > 0) s &= g > 31 ? 0u : ~0u << g;
                seen[c] = s;
                all = all && s == ~0u;
              }
              const bool masked = __any_sync(0xffffffffu, !all);
              float mx = -INFINITY;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                float v[32];
                tmem_ld32(tS + 32 * c, v);
                if (masked) {
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    if (!((seen[c] >> e) & 1u)) v[e] = -INFINITY;
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) mx = fmaxf(mx, v[e]);
              }
              mx *= cf;
              const bool move = mx > m + 6.0f;
              if (__any_sync(0xffffffffu, move && m != -INFINITY)) {
                // rare: O takes the new maximum
                cta_abort.wait(bar(sh.o_full[t]), (no - 1) & 1);
                __syncwarp();
                tc_fence_after();
                const float to = move ? mx : m;
                const float f = m == -INFINITY ? 1.0f : exp2_approx(m - to);
                l *= f;
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                  uint32_t r[16];
                  asm volatile(
                      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,"
                      "%12,%13,%14,%15}, [%16];\n"
                      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                      : "r"(tO + 16 * c));
                  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
                  for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                  tmem_st16(tO + 16 * c, r);
                }
              }
              if (move) m = mx;
              const float mm = m == -INFINITY ? 0.0f : m;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                float v[32];
                tmem_ld32(tS + 32 * c, v);
                if (masked) {
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    if (!((seen[c] >> e) & 1u)) v[e] = -INFINITY;
                }
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  const float p0 = exp2_approx(fmaf(v[e], cf, -mm));
                  const float p1 = exp2_approx(fmaf(v[e + 1], cf, -mm));
                  l += p0 + p1;
                  w[e / 2] = pack_f16x2(p0, p1);
                }
                tmem_st16(tS + 16 * c, w);
              }
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar(sh.p_full[t]));
            ++no;
          }
          // ---- the row of O
          cta_abort.wait(bar(sh.o_full[t]), (no - 1) & 1);
          __syncwarp();
          tc_fence_after();
          uint32_t nan_blocks = 0;  // 16-dimension blocks with a NaN scale at a key of the row
          if (*reinterpret_cast<volatile int*>(&sh.poison)) {
            const int32_t* table = a.page_table + static_cast<long long>(q.b) * a.table_stride;
            const int k0 = max(lo, (q.item.kt0 + q.o) * kPreKeys);
            const int k1 = min(pos, (q.item.kt0 + q.o + q.take) * kPreKeys - 1);
            for (int key = k0; key <= k1; ++key) {
              const int page = __ldg(table + key / a.page_size), in = key % a.page_size;
              if (page < 0 || page >= a.num_pages) continue;
              const uint8_t* at = a.cache + ((static_cast<long long>(page) * a.num_kv_heads + q.h) *
                                                 (a.page_size / 16) + in / 16) * B::kBytes +
                                  B::kVScale + (in % 16) * B::kScaleRow;
              for (int e = 0; e < D / 16; ++e)
                if ((at[e] & 0x7F) == 0x7F) nan_blocks |= 1u << e;
            }
          }
          const bool store = t * 128 + row < live && !cta_abort.raised();
          if (q.take == q.item.nt) {
            const float inv = l == 0.0f ? 0.0f : a.v_scale / l;
            uint16_t* dst = a.out + tok * a.out_stride + head * D;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              float v[32];
              tmem_ld32(tO + 32 * c, v);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                v[e] *= inv;
                if ((nan_blocks >> (2 * c + e / 16)) & 1u) v[e] = __uint_as_float(0x7FC00000u);
              }
              if (store) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                  uint4 w;
                  w.x = pack_t<F16>(v[e], v[e + 1]);
                  w.y = pack_t<F16>(v[e + 2], v[e + 3]);
                  w.z = pack_t<F16>(v[e + 4], v[e + 5]);
                  w.w = pack_t<F16>(v[e + 6], v[e + 7]);
                  *reinterpret_cast<uint4*>(dst + 32 * c + e) = w;
                }
              }
            }
            if (store && a.lse)
              a.lse[static_cast<long long>(tok) * a.num_q_heads + head] =
                  l == 0.0f ? -INFINITY : (m + log2f(l)) * kPreLn2;
          } else {
            const long long slot = static_cast<long long>(blockIdx.x) * 2 + (q.o == 0 ? 1 : 0);
            float* dst = p.part_o + (slot * kPreRows + t * 128 + row) * D;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              float v[32];
              tmem_ld32(tO + 32 * c, v);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if ((nan_blocks >> (2 * c + e / 16)) & 1u) v[e] = __uint_as_float(0x7FC00000u);
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(dst + 32 * c + e) =
                    make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
            }
            p.part_ml[slot * kPreRows + t * 128 + row] = make_float2(m, l);
            __threadfence();
            const int threads = 128 * nact;
            const int w0 = static_cast<int>((q.u - q.o) / per);
            const int w1 = static_cast<int>((q.u - q.o + q.item.nt - 1) / per);
            pre_barrier(nact, threads);
            if (tid == 0) {
              const int last = atomicAdd(p.counters + w0, 1u) == static_cast<uint32_t>(w1 - w0);
              if (last) p.counters[w0] = 0;
              __threadfence();
              sh.last = last;
            }
            pre_barrier(nact, threads);
            if (*reinterpret_cast<volatile int*>(&sh.last)) {
              // every part is there: a warp takes a row at a time, in run order
              const int n = w1 - w0 + 1;
              for (int r = warp; r < live; r += 4 * nact) {
                auto at = [&](int i) {
                  return ((static_cast<long long>(w0) + i) * 2 + (i == 0)) * kPreRows + r;
                };
                float top = -INFINITY;
                for (int i = lane; i < n; i += 32) top = fmaxf(top, __ldcg(&p.part_ml[at(i)]).x);
#pragma unroll
                for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
                float v[D / 32] = {}, sum = 0.0f;
#pragma unroll 4
                for (int i = 0; i < n; ++i) {
                  const float2 ml = __ldcg(&p.part_ml[at(i)]);
                  const float f = ml.x == -INFINITY ? 1.0f : exp2_approx(ml.x - top);
                  sum += ml.y * f;
                  const float* src = p.part_o + at(i) * D + lane * (D / 32);
#pragma unroll
                  for (int e = 0; e < D / 32; e += 2) {
                    const float2 x = __ldcg(reinterpret_cast<const float2*>(src + e));
                    v[e] += x.x * f;
                    v[e + 1] += x.y * f;
                  }
                }
                const int prr = packed0 + r, hh = q.h * group + prr % group;
                const long long tt = q.seq.q0 + prr / group;
                const float inv = sum == 0.0f ? 0.0f : a.v_scale / sum;
                if (!cta_abort.raised()) {
#pragma unroll
                  for (int e = 0; e < D / 32; e += 2)
                    *reinterpret_cast<uint32_t*>(a.out + tt * a.out_stride + hh * D + lane * (D / 32) + e) =
                        pack_t<F16>(v[e] * inv, v[e + 1] * inv);
                  if (lane == 0 && a.lse)
                    a.lse[tt * a.num_q_heads + hh] =
                        sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kPreLn2;
                }
              }
            }
            pre_barrier(nact, threads);  // sh.last may change again
          }
          tc_fence_before();
        }
        stage_it += q.take;
      } while (next_part(q));
    } else if (warp < 12) {
      // -------------------------------------------------------------- keys and values
      const int r = tid - 256;  // key of the tile
      uint4 kc[D / 32], vc[D / 32];
      uint32_t ks[D / 64], vs[D / 64];  // scale bytes
      bool ok = false;
      Part w = q;  // the tile whose loads go out next
      int wj = 0;
      bool more = true;
      auto load = [&]() {
        // codes and scales of this thread's key of tile wj of part w
        const int key = (w.item.kt0 + w.o + wj) * kPreKeys + r;
        ok = key < w.item.hi;
        const uint8_t* blk = nullptr;
        if (ok) {
          const int page = __ldg(a.page_table + static_cast<long long>(w.b) * a.table_stride +
                                 key / a.page_size);
          ok = page >= 0 && page < a.num_pages;
          if (!ok && a.status) atomicOr(a.status, kStatusBadSlot);
          const int in = key % a.page_size;
          blk = a.cache + ((static_cast<long long>(page) * a.num_kv_heads + w.h) * (a.page_size / 16) +
                           in / 16) * B::kBytes;
        }
        if (ok) {
          const int i = key & 15;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            kc[c] = __ldg(reinterpret_cast<const uint4*>(blk + B::kK + i * B::kCodeRow) + c);
            vc[c] = __ldg(reinterpret_cast<const uint4*>(blk + B::kV + i * B::kCodeRow) + c);
          }
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            ks[c] = __ldg(reinterpret_cast<const uint32_t*>(blk + B::kKScale + i * B::kScaleRow) + c);
            vs[c] = __ldg(reinterpret_cast<const uint32_t*>(blk + B::kVScale + i * B::kScaleRow) + c);
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) kc[c] = vc[c] = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) ks[c] = vs[c] = 0;
        }
        if (++wj == w.take) {
          wj = 0;
          more = next_part(w);
        }
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
                make_uint4(pre_hmul2(f[0], s[e / 2]), pre_hmul2(f[1], s[e / 2]),
                           pre_hmul2(f[2], s[e / 2]), pre_hmul2(f[3], s[e / 2]));
          }
        }
      };
      load();
      uint32_t it = 0;
      long long left = u_end - u0;
      for (; left > 0; --left, ++it) {
        const int st = it & 1;
        if (it >= 2) cta_abort.wait(bar(sh.k_empty[st]), ((it >> 1) - 1) & 1);
        __syncwarp();
        const uint32_t votes = __ballot_sync(0xffffffffu, ok);
        put(smem + kOffK + st * kTile, kc, ks);
        if (lane == 0) sh.valid[it & 3][warp - 8] = votes;
        fence_proxy_async();
        __syncwarp();
        mbar_arrive(bar(sh.k_full[st]));
        if (it >= 2) cta_abort.wait(bar(sh.v_empty[st]), ((it >> 1) - 1) & 1);
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
        mbar_arrive(bar(sh.v_full[st]));
        if (more) load();
      }
    } else {
      // -------------------------------------------------------------- products
      uint32_t it = 0, nq[2] = {0, 0}, np[2] = {0, 0};
      auto scores = [&](int t, int st) {
        if (lane == 0 && !cta_abort.raised()) {
          const uint32_t sq = sbase + t * kTile, sk = sbase + kOffK + st * kTile;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * kAtom + (kk & 3) * 32;
            umma_f16(taddr + kColS + t * kPreKeys, umma_desc_sw128(sq + off, 16, 1024),
                     umma_desc_sw128(sk + off, 16, 1024), kIdescS, kk != 0 ? 1u : 0u);
          }
          umma_commit(bar(sh.s_full[t]));
        }
        __syncwarp();
      };
      do {
        const int nact = live_rows(q) > 128 ? 2 : 1;
        for (int t = 0; t < nact; ++t) {
          cta_abort.wait(bar(sh.q_full[t]), nq[t] & 1);
          ++nq[t];
        }
        cta_abort.wait(bar(sh.k_full[it & 1]), (it >> 1) & 1);
        __syncwarp();
        tc_fence_after();
        for (int t = 0; t < nact; ++t) scores(t, it & 1);
        if (lane == 0 && !cta_abort.raised()) umma_commit(bar(sh.k_empty[it & 1]));
        for (int j = 0; j < q.take; ++j, ++it) {
          const int st = it & 1;
          for (int t = 0; t < nact; ++t) {
            cta_abort.wait(bar(sh.p_full[t]), np[t] & 1);
            ++np[t];
            if (t == 0) cta_abort.wait(bar(sh.v_full[st]), (it >> 1) & 1);
            __syncwarp();
            tc_fence_after();
            if (lane == 0 && !cta_abort.raised()) {
              const uint32_t sv = sbase + kOffV + st * kTile;
#pragma unroll
              for (int kk = 0; kk < kPreKeys / 16; ++kk)
                umma_f16_ts(taddr + kColO + t * D, taddr + kColS + t * kPreKeys + 8 * kk,
                            umma_desc_sw128(sv + kk * 16 * 128, kAtom, 1024), kIdescO,
                            (j | kk) != 0 ? 1u : 0u);
              umma_commit(bar(sh.o_full[t]));
              if (t == nact - 1) umma_commit(bar(sh.v_empty[st]));
            }
            __syncwarp();
            if (j + 1 < q.take) {
              const uint32_t nx = it + 1;
              if (t == 0) {
                cta_abort.wait(bar(sh.k_full[nx & 1]), (nx >> 1) & 1);
                __syncwarp();
                tc_fence_after();
              }
              scores(t, nx & 1);
              if (t == nact - 1 && lane == 0 && !cta_abort.raised()) umma_commit(bar(sh.k_empty[nx & 1]));
            }
          }
        }
      } while (next_part(q));
      if (cta_abort.raised()) {  // the products still running end before the TMEM goes
        if (lane == 0) {
          umma_commit(bar(sh.drain));
          mbar_drain(bar(sh.drain), 0, p.wait_limit_ns);
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(kCols)
                 : "memory");
  if (tid == 0 && cta_abort.raised() && a.status) atomicOr(a.status, kStatusTimeout);
}

namespace {
// Sequences of up to kDecodeRows packed rows take the decode kernel, the others
// the prefill kernel; a batch whose bound allows no sequence of a kind does not
// launch that kind's kernel.
constexpr int kDecodeRows = 32;

long long packed_bound(long long max_q_len, int num_q_heads, int num_kv_heads) {
  return max_q_len * (num_q_heads / num_kv_heads);
}
constexpr size_t kPreCounterBytes = 1024;
static_assert(kPreCtasMax * 4 <= kPreCounterBytes, "room for the counters");
size_t prefill_partials(int head_dim) {
  return static_cast<size_t>(2) * kPreCtasMax * kPreRows * (head_dim * 4 + 8);
}
}  // namespace

int launch_kv4_prefill(const Kv4AttnArgs& a, int max_packed_rows, bool f16, cudaStream_t stream) {
  const void* fn =
      a.head_dim == 64 ? (f16 ? reinterpret_cast<const void*>(lora_kv4_prefill_kernel<64, true>)
                              : reinterpret_cast<const void*>(lora_kv4_prefill_kernel<64, false>))
                       : (f16 ? reinterpret_cast<const void*>(lora_kv4_prefill_kernel<128, true>)
                              : reinterpret_cast<const void*>(lora_kv4_prefill_kernel<128, false>));
  const size_t smem = 1024 + 6 * static_cast<size_t>(a.head_dim / 64) * 128 * 128 + sizeof(PreShared);
  if (ensure_smem_attr(fn, smem) != 0) return -6;
  const int sms = device_sm_count();
  if (sms <= 0) return -6;
  PrefillParams p;
  p.a = a;
  char* w = static_cast<char*>(a.workspace);
  p.counters = reinterpret_cast<uint32_t*>(w);
  p.part_o = reinterpret_cast<float*>(w + kPreCounterBytes + kv4_decode_counter_bytes());
  p.part_ml = reinterpret_cast<float2*>(reinterpret_cast<char*>(p.part_o) +
                                        static_cast<size_t>(2) * kPreCtasMax * kPreRows * a.head_dim * 4);
  p.max_packed_rows = max_packed_rows;
  p.wait_fault = wait_fault() ? 1 : 0;
  p.wait_limit_ns = p.wait_fault ? kTestWaitLimitNs : kWaitLimitNs;
  return launch_pdl(fn, dim3(min(sms, kPreCtasMax)), dim3(kPreThreads), smem, stream, 0, &p);
}

// The workspace: the two kernels' counters, then partials, which the kernels of a
// call use one after the other.
size_t kv4_attention_workspace(long long, long long, long long max_q_len, int num_q_heads,
                               int num_kv_heads, int head_dim) {
  const long long packed = packed_bound(max_q_len, num_q_heads, num_kv_heads);
  size_t n = kv4_decode_partial_bytes(packed > 8 ? 16 : 8, head_dim);
  if (packed > kDecodeRows) n = max(n, prefill_partials(head_dim));
  return kPreCounterBytes + kv4_decode_counter_bytes() + n;
}

int launch_kv4_attention(const Kv4AttnArgs& a, bool f16, cudaStream_t stream) {
  const int rc = launch_kv4_decode(a, kDecodeRows, kPreCounterBytes, f16, stream);
  if (rc != 0) return rc;
  return packed_bound(a.max_q_len, a.num_q_heads, a.num_kv_heads) > kDecodeRows
             ? launch_kv4_prefill(a, kDecodeRows, f16, stream)
             : 0;
}

}  // namespace grg
