// Accumulated attention weight of each key of the 4-bit cache:
//   w[j] = (j is one of the rows' own keys ? 0 : w[j]) + sum over rows, heads of exp(x_j - lse)
// from the rows' logarithms of sums that the attention has left, so that one pass over K
// forms them: no maximum, no sum over keys, nothing to join.
//
// For a block of 16 keys and 8 * NT packed rows (mma.sync m16n8k16, fp16 operands, fp32
// accumulators): S = K Q^T as in the decode attention, p = 2^(S c - lse log2 e), summed over
// the rows in the lanes of a key.  A warp takes a run of the line of all blocks of all
// (sequence, key head), cut into equal runs whatever the lengths; a key's sum is one warp's,
// in the rows' order, so results do not depend on the cut.
//
// Measured (GB300, bf16): 256 sequences of one row over up to 4096 keys, 32 / 8 heads of 128 (K's
// half of the cache and the weights, 338 MB): 89 us, 0.56 of measured HBM; of heads of 64 66 us; one
// sequence of 700 keys 4.4 us.  Bound by latencies at 16 warps an SM: some 200 instructions a block
// of 16 keys fill 54 % of the issue slots (four blocks' codes in flight take the registers that a
// third CTA would need); a ring of bulk copies in place of the loads 90.1 us.  One sequence:
// lengths, line, page, codes, weights, one after the other.
#include "kv4_weights.cuh"
#include "launch.h"

namespace grg {

namespace {
constexpr int kWtsWarps = 8, kWtsThreads = kWtsWarps * 32;
constexpr int kWtsBatch = 4;  // blocks whose codes are asked for together
// CTAs of an SM (256 sequences of up to 4096 keys, heads of 128: 89 us by two of 4 blocks, 110 us of 2,
// 102 us by three; of 64: 73 us by two, 66 us by three).
template <int D>
constexpr int kWtsCtas = D == 64 ? 3 : 2;
constexpr float kWtsLog2e = 1.4426950408889634f;

struct WtsParams {
  Kv4WeightsArgs a;
  int max_packed_rows;  // sequences with more packed rows are not this kernel's
};
__device__ __forceinline__ uint32_t wts_both(uint32_t a, bool high) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %1, %2;\n" : "=r"(r) : "r"(a), "r"(high ? 0x3232u : 0x1010u));
  return r;
}
}  // namespace

template <int D, int NT, bool F16>
__global__ void __launch_bounds__(kWtsThreads, kWtsCtas<D>)
    lora_kv4_weights_kernel(const __grid_constant__ WtsParams p) {
  using B = Kv4Block<D>;
  constexpr int KS = D / 16, ROWS = 8 * NT, W = D / 32;  // W: words of a thread's codes of a key
  __shared__ long long s_prefix[kWtsThreads + 1], s_warp[kWtsWarps];
  const Kv4WeightsArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int group = a.num_q_heads / a.num_kv_heads;
  pdl_wait();
  pdl_launch_dependents();

  // ---- the line of blocks
  auto blocks_of = [&](const WeightSeq& s) {
    return static_cast<long long>(s.take) * group > p.max_packed_rows ? 0 : s.blocks(a.window);
  };
  const int per_thread = (a.num_seqs + kWtsThreads - 1) / kWtsThreads;
  long long mine = 0;
  for (int i = 0; i < per_thread; ++i) {
    const int b = tid * per_thread + i;
    if (b < a.num_seqs) {
      const WeightSeq s = WeightSeq::of(a, b);
      if (s.odd && blockIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadLength);
      mine += static_cast<long long>(blocks_of(s)) * a.num_kv_heads;
    }
  }
  long long run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += v;
  }
  if (lane == 31) s_warp[warp] = run;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWtsWarps; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  s_prefix[tid] = before + run - mine;
  __syncthreads();
  const long long workers = static_cast<long long>(gridDim.x) * kWtsWarps;
  const long long per = quotient(all + workers - 1, workers);
  const long long u0 = (static_cast<long long>(blockIdx.x) * kWtsWarps + warp) * per;
  long long left = min(per, all - u0);
  if (left <= 0) return;

  // ---- the first place: sequence b, head h, block o of the head's
  int b, h, o, nb;
  WeightSeq seq;
  {
    const int lo = last_not_past<kWtsWarps>(s_prefix, u0, lane);
    long long off = u0 - s_prefix[lo];
    for (b = lo * per_thread;; ++b) {
      seq = WeightSeq::of(a, b);
      nb = blocks_of(seq);
      const long long n = static_cast<long long>(nb) * a.num_kv_heads;
      if (off < n) break;
      off -= n;
    }
    h = static_cast<int>(quotient(off, nb));
    o = static_cast<int>(off - static_cast<long long>(h) * nb);
  }
  const int page_blocks = a.page_size / 16;
  bool lost = false, odd = false;
  while (true) {
    const int take = static_cast<int>(min(static_cast<long long>(nb - o), left));
    const int blk0 = seq.first_block(a.window) + o;
    const int packed = seq.take * group;
    const int32_t* table = a.page_table + b * a.table_stride;
    float* wrow = a.weights + (static_cast<long long>(b) * a.num_kv_heads + h) * a.capacity;
    const int fresh = max(seq.kv - seq.rows, 0);  // from this key on weights begin at 0
    for (int row0 = 0; row0 == 0 || row0 < packed; row0 += ROWS) {
      // ---- the rows' queries as B fragments in fp16, their factors and logarithms
      uint32_t qf[NT][KS][2];
      float cf[NT][2], sub[NT][2];
      int pos[NT][2], lo[NT][2];
      int pos_min = 0x7fffffff, lo_max = 0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float v[KS * 4], top = 0.0f;
        const int r = row0 + nt * 8 + g;
        int at = -1, head = 0, i = 0;
        if (r < packed) {
          i = r / group;
          head = h * group + r - i * group;
          at = seq.row_in_q(a, b, i);
          if (at < 0) odd = true;
        }
        const uint16_t* src = a.q + at * a.q_stride + head * D + t4 * (D / 4);
#pragma unroll
        for (int c = 0; c < KS / 2; ++c) {
          const uint4 raw = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
          const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = unpack_t<F16>(x[k]);
            v[8 * c + 2 * k] = f.x, v[8 * c + 2 * k + 1] = f.y;
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
        float lse = at >= 0 ? __ldg(a.lse + static_cast<long long>(at) * a.num_q_heads + head) : -INFINITY;
        const bool adds = lse != -INFINITY;
        lse = adds ? lse * kWtsLog2e : INFINITY;  // (2^-infinity is 0)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float up, down;
        row_factor(top, up, down);
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          qf[nt][j][0] = pack_f16x2(v[4 * j] * up, v[4 * j + 1] * up);
          qf[nt][j][1] = pack_f16x2(v[4 * j + 2] * up, v[4 * j + 3] * up);
        }
        // What adds nothing sees nothing, a row without lse or what lies behind the last row: no
        // key of NaN makes it one.
        const int my_pos = r < packed && adds ? seq.pos(i) : -1;
        const int in_window = seq.first_key(i, a.window), my_lo = a.path ? min(in_window, fresh) : in_window;
        if (r < packed) pos_min = min(pos_min, my_pos), lo_max = max(lo_max, my_lo);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int from = (2 * t4 + c) * 4;  // the thread's columns of S are rows 2 t4 and 2 t4 + 1
          cf[nt][c] = score_factor(__shfl_sync(0xffffffffu, down, from), a.score_scale * kWtsLog2e);
          sub[nt][c] = __shfl_sync(0xffffffffu, lse, from);
          pos[nt][c] = __shfl_sync(0xffffffffu, my_pos, from);
          lo[nt][c] = __shfl_sync(0xffffffffu, my_lo, from);
        }
      }
      pos_min = __reduce_min_sync(0xffffffffu, pos_min);
      lo_max = __reduce_max_sync(0xffffffffu, lo_max);

      const unsigned char* addr = nullptr;  // lane l holds that of block (i & ~31) + l
      for (int i = 0; i < take; i += kWtsBatch) {
        if ((i & 31) == 0) {
          addr = nullptr;
          if (i + lane < take) {
            const int blk = blk0 + i + lane, pg = blk / page_blocks, page = __ldg(table + pg);
            if (page >= 0 && page < a.num_pages)
              addr = a.cache + ((static_cast<long long>(page) * a.num_kv_heads + h) * page_blocks +
                                (blk - pg * page_blocks)) * B::kBytes;
            else lost = true;
          }
        }
        uint32_t ca[kWtsBatch][W], cb[kWtsBatch][W];
        uint32_t ea[kWtsBatch], eb[kWtsBatch];
        float old[kWtsBatch];
        uint32_t have = 0;
#pragma unroll
        for (int u = 0; u < kWtsBatch; ++u) {
          const unsigned char* blk = reinterpret_cast<const unsigned char*>(__shfl_sync(
              0xffffffffu, reinterpret_cast<unsigned long long>(addr), (i + u) & 31));
          if (i + u >= take) blk = nullptr;
#pragma unroll
          for (int w = 0; w < W; ++w) ca[u][w] = cb[u][w] = 0;
          ea[u] = eb[u] = 0;
          old[u] = 0.0f;
          if (blk) {
            have |= 1u << u;
            if constexpr (D == 128) {
              const uint4 va = __ldg(reinterpret_cast<const uint4*>(blk + g * 64 + 16 * t4));
              const uint4 vb = __ldg(reinterpret_cast<const uint4*>(blk + (g + 8) * 64 + 16 * t4));
              ca[u][0] = va.x, ca[u][1] = va.y, ca[u][2] = va.z, ca[u][3] = va.w;
              cb[u][0] = vb.x, cb[u][1] = vb.y, cb[u][2] = vb.z, cb[u][3] = vb.w;
              ea[u] = __ldg(reinterpret_cast<const uint16_t*>(blk + B::kKScale + g * 8 + 2 * t4));
              eb[u] = __ldg(reinterpret_cast<const uint16_t*>(blk + B::kKScale + (g + 8) * 8 + 2 * t4));
            } else {
              const uint2 va = __ldg(reinterpret_cast<const uint2*>(blk + g * 32 + 8 * t4));
              const uint2 vb = __ldg(reinterpret_cast<const uint2*>(blk + (g + 8) * 32 + 8 * t4));
              ca[u][0] = va.x, ca[u][1] = va.y, cb[u][0] = vb.x, cb[u][1] = vb.y;
              ea[u] = __ldg(blk + B::kKScale + g * 4 + t4);
              eb[u] = __ldg(blk + B::kKScale + (g + 8) * 4 + t4);
            }
          }
          const int j = 16 * (blk0 + i + u) + g + 8 * t4;  // (of lanes with t4 below 2)
          if (t4 < 2 && i + u < take && j < seq.end && (j < fresh || row0 > 0)) old[u] = wrow[j];
        }
#pragma unroll
        for (int u = 0; u < kWtsBatch; ++u) {
          if (i + u >= take) break;
          const int tok = 16 * (blk0 + i + u);
          float sc[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[nt][c] = 0.0f;
          const uint32_t ha = e4m3x2_to_f16(ea[u]), hb = e4m3x2_to_f16(eb[u]);
#pragma unroll
          for (int w = 0; w < W; ++w) {
            uint32_t fa[4], fb[4];
            e2m1x8_to_f16(ca[u][w], fa);
            e2m1x8_to_f16(cb[u][w], fb);
            const uint32_t xa = wts_both(ha, D == 128 && w >= 2), xb = wts_both(hb, D == 128 && w >= 2);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t frag[4] = {hmul2(fa[2 * j], xa), hmul2(fb[2 * j], xb),
                                        hmul2(fa[2 * j + 1], xa), hmul2(fb[2 * j + 1], xb)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(sc[nt], frag, qf[nt][2 * w + j][0], qf[nt][2 * w + j][1]);
            }
          }
          const bool masked = tok + 15 > pos_min || tok < lo_max || !((have >> u) & 1u);
          float sum[2] = {0.0f, 0.0f};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float x = exp2_approx(fmaf(sc[nt][c], cf[nt][c & 1], -sub[nt][c & 1]));
              if (masked) {
                const int j = tok + g + 8 * (c >> 1);
                if (j > pos[nt][c & 1] || j < lo[nt][c & 1] || !((have >> u) & 1u)) x = 0.0f;
              }
              sum[c >> 1] += x;
            }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], 1);
            sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], 2);
          }
          const int j = tok + g + 8 * t4;
          if (t4 < 2 && j < seq.end) wrow[j] = old[u] + (t4 ? sum[1] : sum[0]);
        }
      }
    }
    left -= take;
    if (left == 0) break;
    o = 0;
    if (++h == a.num_kv_heads) {
      h = 0;
      do {
        seq = WeightSeq::of(a, ++b);
        nb = blocks_of(seq);
      } while (nb == 0);
    }
  }
  if (a.status) {
    if (odd) atomicOr(a.status, kStatusBadLength);
    if (lost) atomicOr(a.status, kStatusBadSlot);
  }
}

namespace {
template <int D, bool F16>
int run_weights(const WtsParams& q, bool wide, cudaStream_t stream) {
  WtsParams p = q;
  const void* fn = wide ? reinterpret_cast<const void*>(lora_kv4_weights_kernel<D, 2, F16>)
                        : reinterpret_cast<const void*>(lora_kv4_weights_kernel<D, 1, F16>);
  const int sms = device_sm_count();
  if (sms <= 0) return -6;
  return launch_pdl(fn, dim3(kWtsCtas<D> * sms), dim3(kWtsThreads), 0, stream, 0, &p);
}
}  // namespace

// Sequences of up to kFewRows packed rows go by mma.sync, the others by tcgen05 (64 sequences of
// 2000 keys, 32 / 8 heads of 128: of 16 packed rows 33 us by mma.sync, of 32 57, of 36 80, of 64 105 us;
// by tcgen05 72 us up to a tile of 128 rows); a batch whose bound allows no long sequence does
// not launch the latter.
constexpr int kFewRows = 32;

int launch_kv4_weights(const Kv4WeightsArgs& a, bool f16, cudaStream_t stream) {
  const long long packed = static_cast<long long>(a.max_q_len) * (a.num_q_heads / a.num_kv_heads);
  WtsParams p;
  p.a = a;
  p.max_packed_rows = kFewRows;
  const int rc = a.head_dim == 64 ? (f16 ? run_weights<64, true>(p, packed > 8, stream) : run_weights<64, false>(p, packed > 8, stream))
                                  : (f16 ? run_weights<128, true>(p, packed > 8, stream) : run_weights<128, false>(p, packed > 8, stream));
  return rc == 0 && packed > kFewRows ? launch_kv4_weights_tc(a, kFewRows, f16, stream) : rc;
}

}  // namespace grg
