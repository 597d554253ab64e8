// Rotation of q and k by position and the append of k and v to the 4-bit
// paged cache (layout in kv4.cuh).  One thread per two blocks of 16 dimensions
// (the unit of a scale) of one head of one token: the two blocks that rotate
// against each other in the half-split form, so q may be rotated in place.
// Everything is computed in fp32 with each product, sum and quotient rounded
// once, so the stored codes and scales are those of the definition in fp32,
// bit for bit.
#include "kv4.cuh"
#include "launch.h"
#include "layer.h"

namespace grg {

namespace {
// Measured on 8000 tokens of 32 q and 8 kv heads (210 MB, 0.76 of measured HBM): 40.5 us with
// CTAs of 64 threads, 41.1 us of 96, 44.3 us of 192 (8192 tokens of 64 and 8 heads: 66.3,
// 70.6 and 75.9 us), all with 80 registers a thread (16 bytes spilled); with 64 registers
// 41.9 us, and 61.2 us on the second case, but 5.2 against 4.3 us for 256 tokens.
constexpr int kAppendThreads = 128;
constexpr int kAppendCtas = 6;

struct AppendParams {
  Kv4AppendArgs a;
  int tokens;  // of a CTA
  int ctas;    // of a token
};

struct RawBlock {
  uint4 w[2];
  __device__ __forceinline__ void load(const uint16_t* src) {
    w[0] = reinterpret_cast<const uint4*>(src)[0];
    w[1] = reinterpret_cast<const uint4*>(src)[1];
  }
};
template <bool F16>
__device__ __forceinline__ void unpack_block(const RawBlock& raw, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 w = raw.w[i];
    const float2 a = unpack_t<F16>(w.x), b = unpack_t<F16>(w.y), c = unpack_t<F16>(w.z),
                 d = unpack_t<F16>(w.w);
    v[8 * i + 0] = a.x, v[8 * i + 1] = a.y, v[8 * i + 2] = b.x, v[8 * i + 3] = b.y;
    v[8 * i + 4] = c.x, v[8 * i + 5] = c.y, v[8 * i + 6] = d.x, v[8 * i + 7] = d.y;
  }
}
template <bool F16>
__device__ __forceinline__ void store_block(uint16_t* dst, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint4 w;
    w.x = pack_t<F16>(v[8 * i + 0], v[8 * i + 1]);
    w.y = pack_t<F16>(v[8 * i + 2], v[8 * i + 3]);
    w.z = pack_t<F16>(v[8 * i + 4], v[8 * i + 5]);
    w.w = pack_t<F16>(v[8 * i + 6], v[8 * i + 7]);
    reinterpret_cast<uint4*>(dst)[i] = w;
  }
}
}  // namespace

// The larger one, or NaN where one is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Quantises one block and stores its codes (and, when asked, what it then stands
// for); returns the scale byte.
template <bool F16>
__device__ __forceinline__ uint32_t append_block(float (&v)[16], float factor, float inv,
                                                 uint8_t* codes, uint16_t* held) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = __fmul_rn(v[i], inv);
    top = max_nan(top, fabsf(v[i]));
  }
  const uint32_t s8 = f32x2_to_e4m3(__fdiv_rn(top, 6.0f), 0.0f) & 0xFFu;
  const float scale = e4m3_to_f32(s8);
  uint32_t code[2] = {0, 0};
  if (scale > 0.0f) {
    // Quotients v / scale, correctly rounded (Markstein, 1990: with the correctly
    // rounded reciprocal r, q - (q scale - v) r rounds to the quotient's nearest
    // where q = v r; in this order of the signs -0 stays -0).  At the largest scale v
    // may be as large as infinity: what is beyond 6 * 448 becomes 6 either way.
    const float r = __frcp_rn(scale);
    if (s8 == 0x7Eu) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = fminf(fmaxf(v[i], -4096.0f), 4096.0f);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float q = __fmul_rn(v[i], r);
      v[i] = __fmaf_rn(-__fmaf_rn(q, scale, -v[i]), r, q);
    }
    code[0] = f32x8_to_e2m1(v);
    code[1] = f32x8_to_e2m1(v + 8);
  }
  *reinterpret_cast<uint2*>(codes) = make_uint2(code[0], code[1]);
  if (held) {
    uint32_t h[2][4];
    e2m1x8_to_f16(code[0], h[0]);
    e2m1x8_to_f16(code[1], h[1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = unpack_f16x2(h[i / 4][i % 4]);
      v[2 * i] = __fmul_rn(__fmul_rn(f.x, scale), factor);
      v[2 * i + 1] = __fmul_rn(__fmul_rn(f.y, scale), factor);
    }
    store_block<F16>(held, v);
  }
  return s8;
}

// Unit u of token t: two blocks of one head.
template <int D, bool F16>
__device__ __forceinline__ void append_pair(const Kv4AppendArgs& p, int t, int u) {
  using B = Kv4Block<D>;
  constexpr int kPairs = D / 32;
  const int head = u / kPairs, pair = u % kPairs;
  // which of q, k and v, and the head within it
  const int kind = head < p.num_q_heads ? 0 : head < p.num_q_heads + p.num_kv_heads ? 1 : 2;
  const int hh = kind == 0 ? head : kind == 1 ? head - p.num_q_heads
                                              : head - p.num_q_heads - p.num_kv_heads;
  const uint16_t* row = (kind == 0 ? p.q + t * p.q_stride
                                   : kind == 1 ? p.k + t * p.k_stride : p.v + t * p.v_stride) +
                        hh * D;
  // blocks that rotate against each other, or two that stay as they are
  const int turning = p.rope ? p.rope_dim / 32 : kPairs;
  const int b0 = pair < turning ? pair : 2 * pair, b1 = pair < turning ? pair + turning : b0 + 1;
  // everything whose address is known goes out at once; a row past n is loaded
  // and dropped
  RawBlock r0, r1;
  r0.load(row + 16 * b0);
  r1.load(row + 16 * b1);
  const int raw = *p.num_tokens;
  const int pos = p.rope ? p.positions[t] : 0, slot = p.slots[t];
  const int n = min(max(raw, 0), p.max_num_tokens);
  if (raw != n && p.status && t == 0 && u == 0) atomicOr(p.status, kStatusBadNumTokens);
  if (t >= n) return;
  if (p.rope && (pos < 0 || pos >= p.max_positions)) {
    if (p.status && u == 0) atomicOr(p.status, kStatusBadPosition);
    return;
  }
  if (kind != 0 && (slot < 0 || slot >= p.num_slots)) {
    if (slot != -1 && p.status) atomicOr(p.status, kStatusBadSlot);
    return;
  }
  float lo[16], hi[16];
  unpack_block<F16>(r0, lo);
  unpack_block<F16>(r1, hi);
  if (kind != 2 && p.rope && pair < turning) {
    const int half = p.rope_dim / 2;
    const float* table = p.rope + static_cast<long long>(pos) * p.rope_dim;
    auto turn = [](float& x, float& y, float c, float s) {
      const float x0 = x;
      x = __fsub_rn(__fmul_rn(x0, c), __fmul_rn(y, s));
      y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x0, s));
    };
    auto angles = [&](int at, float (&c)[4], float (&s)[4]) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(table + at));
      const float4 b = __ldg(reinterpret_cast<const float4*>(table + half + at));
      c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
      s[0] = b.x, s[1] = b.y, s[2] = b.z, s[3] = b.w;
    };
    float c[4], s[4];
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        angles(8 * b0 + i, c, s);
#pragma unroll
        for (int e = 0; e < 4; ++e) turn(lo[2 * (i + e)], lo[2 * (i + e) + 1], c[e], s[e]);
        angles(8 * b1 + i, c, s);
#pragma unroll
        for (int e = 0; e < 4; ++e) turn(hi[2 * (i + e)], hi[2 * (i + e) + 1], c[e], s[e]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        angles(16 * b0 + i, c, s);
#pragma unroll
        for (int e = 0; e < 4; ++e) turn(lo[i + e], hi[i + e], c[e], s[e]);
      }
    }
  }
  if (kind == 0) {
    uint16_t* o = p.q_out + t * p.q_out_stride + hh * D;
    store_block<F16>(o + 16 * b0, lo);
    store_block<F16>(o + 16 * b1, hi);
    return;
  }
  const float factor = kind == 1 ? p.k_scale : p.v_scale;
  const float inv = kind == 1 ? p.inv_k_scale : p.inv_v_scale;
  const int page = slot / p.page_size, in = slot % p.page_size, r = in % 16;
  uint8_t* blk = p.cache + ((static_cast<long long>(page) * p.num_kv_heads + hh) *
                                (p.page_size / 16) + in / 16) * B::kBytes;
  uint8_t* codes = blk + (kind == 1 ? B::kK : B::kV) + r * B::kCodeRow;
  uint8_t* scales = blk + (kind == 1 ? B::kKScale : B::kVScale) + r * B::kScaleRow;
  uint16_t* held = kind == 1 ? p.k_held : p.v_held;
  if (held) held += (static_cast<long long>(t) * p.num_kv_heads + hh) * D;
  const uint32_t s0 =
      append_block<F16>(lo, factor, inv, codes + 8 * b0, held ? held + 16 * b0 : held);
  const uint32_t s1 =
      append_block<F16>(hi, factor, inv, codes + 8 * b1, held ? held + 16 * b1 : held);
  // the head's threads (neighbouring lanes) join their scale bytes into one store
  unsigned long long all = (static_cast<unsigned long long>(s0) << (8 * b0)) |
                           (static_cast<unsigned long long>(s1) << (8 * b1));
  const uint32_t group = ((1u << kPairs) - 1u) << ((threadIdx.x & 31) & ~(kPairs - 1));
#pragma unroll
  for (int o = 1; o < kPairs; o <<= 1) all |= __shfl_xor_sync(group, all, o);
  if (pair == 0) {
    if constexpr (D == 128) *reinterpret_cast<unsigned long long*>(scales) = all;
    else *reinterpret_cast<uint32_t*>(scales) = static_cast<uint32_t>(all);
  }
}

// One unit (append_pair) per thread: several tokens in a CTA of up to 128 threads where a
// token has few units, else one or more CTAs a token.
template <int D, bool F16>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas)
    lora_kv4_append_kernel(const AppendParams q) {
  const Kv4AppendArgs& p = q.a;
  const int tokens = q.tokens, ctas = q.ctas;
  const int per = (p.num_q_heads + 2 * p.num_kv_heads) * (D / 32);  // units of one token
  int t, u;
  if (tokens > 1) {
    const int in = static_cast<int>(threadIdx.x) / per;
    t = in < tokens ? blockIdx.x * tokens + in : p.max_num_tokens;
    u = threadIdx.x - in * per;
  } else {
    t = blockIdx.x / ctas;
    u = (blockIdx.x - t * ctas) * blockDim.x + threadIdx.x;
  }
  pdl_wait();
  pdl_launch_dependents();
  if (t < p.max_num_tokens && u < per) append_pair<D, F16>(p, t, u);
}

int launch_kv4_append(const Kv4AppendArgs& a, bool f16, cudaStream_t stream) {
  const void* fn =
      a.head_dim == 64 ? (f16 ? reinterpret_cast<const void*>(lora_kv4_append_kernel<64, true>)
                              : reinterpret_cast<const void*>(lora_kv4_append_kernel<64, false>))
                       : (f16 ? reinterpret_cast<const void*>(lora_kv4_append_kernel<128, true>)
                              : reinterpret_cast<const void*>(lora_kv4_append_kernel<128, false>));
  const int per = (a.num_q_heads + 2 * a.num_kv_heads) * (a.head_dim / 32);
  // a token of up to 64 units shares its CTA; else the CTA size that leaves the fewest
  // threads idle, the smallest of them (small CTAs come and go more evenly)
  int tokens = 1, ctas = 1, threads;
  if (per <= 64) {
    tokens = kAppendThreads / per;
    threads = (per * tokens + 31) / 32 * 32;
  } else {
    threads = 64;
    for (int x = 96; x <= kAppendThreads; x += 32)
      if ((per + x - 1) / x * x < (per + threads - 1) / threads * threads) threads = x;
    ctas = (per + threads - 1) / threads;
  }
  const long long grid = tokens > 1 ? (a.max_num_tokens + tokens - 1) / tokens
                                    : static_cast<long long>(a.max_num_tokens) * ctas;
  if (grid > 0x7FFFFFFFll) return -3;
  AppendParams p{a, tokens, ctas};
  return launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(threads), 0, stream, 0, &p);
}

}  // namespace grg
