// Attention over the 4-bit paged cache (layout in kv4.cuh) for sequences with
// many query rows: one warp per row and head walks the row's keys once, with the
// running maximum and sum of the softmax in fp32.
#include "kv4_attention.cuh"
#include "kv4_attention.h"
#include "launch.h"

namespace grg {

namespace {
constexpr int kAttnThreads = 128;

// The sequence of row t: the last b with q_start[b] <= t.
__device__ __forceinline__ int seq_of(const int32_t* q_start, int num_seqs, int t) {
  int lo = 0, hi = num_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (q_start[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}
}  // namespace

namespace {
struct PrefillParams {
  Kv4AttnArgs a;
  int max_packed_rows;
};
}  // namespace

template <int D, bool F16>
__global__ void __launch_bounds__(kAttnThreads) lora_kv4_prefill_kernel(const PrefillParams pp) {
  const Kv4AttnArgs& p = pp.a;
  const int max_packed_rows = pp.max_packed_rows;
  using B = Kv4Block<D>;
  constexpr int E = D / 32;  // dimensions of a lane
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long id =
      (static_cast<long long>(blockIdx.x) * kAttnThreads + threadIdx.x) / 32;
  const int t = static_cast<int>(id / p.num_q_heads), h = static_cast<int>(id % p.num_q_heads);
  const int end = p.q_start[p.num_seqs];
  if (t >= min(end, p.max_num_tokens)) return;
  const int b = seq_of(p.q_start, p.num_seqs, t);
  const Kv4Seq seq = Kv4Seq::of(p, b);
  if (t < seq.q0 || t - seq.q0 >= seq.take ||
      static_cast<long long>(seq.take) * (p.num_q_heads / p.num_kv_heads) <= max_packed_rows)
    return;
  const int kv = seq.kv, pos = seq.pos(t - seq.q0), first = seq.first_key(t - seq.q0, p.window);
  const int kvh = h / (p.num_q_heads / p.num_kv_heads);
  float q[E], acc[E], top = -INFINITY, sum = 0.0f;
  const uint16_t* qr = p.q + t * p.q_stride + h * D + lane * E;
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    const float2 f = unpack_t<F16>(*reinterpret_cast<const uint32_t*>(qr + i));
    q[i] = f.x, q[i + 1] = f.y;
    acc[i] = acc[i + 1] = 0.0f;
  }
  for (int j = first; j <= min(pos, kv - 1); ++j) {
    const int page = p.page_table[b * p.table_stride + j / p.page_size];
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0 && p.status) atomicOr(p.status, kStatusBadSlot);
      continue;
    }
    const int in = j % p.page_size;
    const uint8_t* blk = p.cache + ((static_cast<long long>(page) * p.num_kv_heads + kvh) *
                                        (p.page_size / 16) + in / 16) * B::kBytes;
    const int r = in % 16;
    float k[E], v[E];
    auto take = [&](int codes, int scales, float (&o)[E]) {
      const uint8_t* c = blk + codes + r * B::kCodeRow + lane * E / 2;
      const float s = e4m3_to_f32(blk[scales + r * B::kScaleRow + lane * E / 16]);
      uint32_t f[4];
      e2m1x8_to_f16(E == 4 ? *reinterpret_cast<const uint16_t*>(c) : *c, f);
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const float2 g = unpack_f16x2(f[i / 2]);
        o[i] = g.x * s, o[i + 1] = g.y * s;
      }
    };
    take(B::kK, B::kKScale, k);
    take(B::kV, B::kVScale, v);
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) x += q[i] * k[i];
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    x *= p.score_scale;
    const float now = fmaxf(top, x);
    const float keep = now == -INFINITY ? 0.0f : expf(top - now);
    const float e = now == -INFINITY ? 0.0f : expf(x - now);
    sum = sum * keep + e;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = acc[i] * keep + e * v[i];
    top = now;
  }
  const float inv = sum > 0.0f ? p.v_scale / sum : (sum == 0.0f ? 0.0f : sum);
  uint16_t* o = p.out + t * p.out_stride + h * D + lane * E;
#pragma unroll
  for (int i = 0; i < E; i += 2)
    *reinterpret_cast<uint32_t*>(o + i) = pack_t<F16>(acc[i] * inv, acc[i + 1] * inv);
  if (p.lse && lane == 0)
    p.lse[static_cast<long long>(t) * p.num_q_heads + h] = sum > 0.0f ? top + logf(sum) : sum == 0.0f ? -INFINITY : sum;
}


int launch_kv4_prefill(const Kv4AttnArgs& a, int max_packed_rows, bool f16, cudaStream_t stream) {
  const void* fn =
      a.head_dim == 64 ? (f16 ? reinterpret_cast<const void*>(lora_kv4_prefill_kernel<64, true>)
                              : reinterpret_cast<const void*>(lora_kv4_prefill_kernel<64, false>))
                       : (f16 ? reinterpret_cast<const void*>(lora_kv4_prefill_kernel<128, true>)
                              : reinterpret_cast<const void*>(lora_kv4_prefill_kernel<128, false>));
  const long long warps = static_cast<long long>(a.max_num_tokens) * a.num_q_heads;
  const long long grid = (warps * 32 + kAttnThreads - 1) / kAttnThreads;
  if (grid > 0x7FFFFFFFll) return -3;
  PrefillParams p{a, max_packed_rows};
  return launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(kAttnThreads), 0, stream, 0, &p);
}

// Sequences of up to kDecodeRows packed rows take the decode kernel, the others
// the prefill kernel; a batch whose bound allows no sequence of a kind does not
// launch that kind's kernel.
constexpr int kDecodeRows = 32;

size_t kv4_attention_workspace(long long, long long, long long max_q_len, int num_q_heads,
                               int num_kv_heads, int head_dim) {
  return kv4_decode_workspace(max_q_len * (num_q_heads / num_kv_heads) > 8 ? 16 : 8, head_dim);
}

int launch_kv4_attention(const Kv4AttnArgs& a, bool f16, cudaStream_t stream) {
  const int rc = launch_kv4_decode(a, kDecodeRows, f16, stream);
  if (rc != 0) return rc;
  const long long packed = static_cast<long long>(a.max_q_len) * (a.num_q_heads / a.num_kv_heads);
  return packed > kDecodeRows ? launch_kv4_prefill(a, kDecodeRows, f16, stream) : 0;
}

}  // namespace grg
