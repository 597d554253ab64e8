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
constexpr int kAppendThreads = 256;

template <bool F16>
__device__ __forceinline__ void load_block(const uint16_t* src, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 w = reinterpret_cast<const uint4*>(src)[i];
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

// Quantises one block and stores it (and, when asked, what it then stands for).
template <int D, bool F16>
__device__ __forceinline__ void append_block(float (&v)[16], float factor, float inv, uint8_t* codes,
                                             uint8_t* scales, uint16_t* held) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = __fmul_rn(v[i], inv);
    top = max(top, abs_bits(v[i]));
  }
  const uint32_t s8 = f32x2_to_e4m3(__fdiv_rn(__uint_as_float(top), 6.0f), 0.0f) & 0xFFu;
  const float scale = e4m3_to_f32(s8);
  uint32_t code[2] = {0, 0};
  if (scale > 0.0f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __fdiv_rn(v[i], scale);
    code[0] = f32x8_to_e2m1(v);
    code[1] = f32x8_to_e2m1(v + 8);
  }
  *reinterpret_cast<uint2*>(codes) = make_uint2(code[0], code[1]);
  *scales = static_cast<uint8_t>(s8);
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
}

template <int D, bool F16>
__global__ void __launch_bounds__(kAppendThreads) lora_kv4_append_kernel(const Kv4AppendArgs p) {
  using B = Kv4Block<D>;
  constexpr int kPairs = D / 32;
  pdl_wait();
  pdl_launch_dependents();
  const int raw = *p.num_tokens;
  const int n = min(max(raw, 0), p.max_num_tokens);
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  const int per = heads * kPairs;  // threads of one token
  const long long id = static_cast<long long>(blockIdx.x) * kAppendThreads + threadIdx.x;
  const int t = static_cast<int>(id / per);
  if (raw != n && p.status && id == 0) atomicOr(p.status, kStatusBadNumTokens);
  if (t >= n) return;
  const int u = static_cast<int>(id % per);
  const int head = u / kPairs, pair = u % kPairs;
  // which of q, k and v, and the head within it
  const int kind = head < p.num_q_heads ? 0 : head < p.num_q_heads + p.num_kv_heads ? 1 : 2;
  const int hh = kind == 0 ? head : kind == 1 ? head - p.num_q_heads
                                              : head - p.num_q_heads - p.num_kv_heads;
  int pos = 0, slot = 0;
  if (p.rope) {
    pos = p.positions[t];
    if (pos < 0 || pos >= p.max_positions) {
      if (p.status && u == 0) atomicOr(p.status, kStatusBadPosition);
      return;
    }
  }
  if (kind != 0) {
    slot = p.slots[t];
    if (slot < 0 || slot >= p.num_slots) {
      if (slot != -1 && p.status) atomicOr(p.status, kStatusBadSlot);
      return;
    }
  }
  const uint16_t* row = (kind == 0 ? p.q + t * p.q_stride
                                   : kind == 1 ? p.k + t * p.k_stride : p.v + t * p.v_stride) +
                        hh * D;
  // blocks that rotate against each other, or two that stay as they are
  const int turning = p.rope ? p.rope_dim / 32 : kPairs;
  const int b0 = pair < turning ? pair : 2 * pair, b1 = pair < turning ? pair + turning : b0 + 1;
  float lo[16], hi[16];
  load_block<F16>(row + 16 * b0, lo);
  load_block<F16>(row + 16 * b1, hi);
  if (kind != 2 && p.rope && pair < turning) {
    const int half = p.rope_dim / 2;
    const float* table = p.rope + static_cast<long long>(pos) * p.rope_dim;
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        auto turn = [&](float& a, float& b, int at) {
          const float c = __ldg(table + at), s = __ldg(table + half + at), a0 = a;
          a = __fsub_rn(__fmul_rn(a0, c), __fmul_rn(b, s));
          b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a0, s));
        };
        turn(lo[2 * i], lo[2 * i + 1], 8 * b0 + i);
        turn(hi[2 * i], hi[2 * i + 1], 8 * b1 + i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float c = __ldg(table + 16 * b0 + i), s = __ldg(table + half + 16 * b0 + i);
        const float a = lo[i], b = hi[i];
        lo[i] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
        hi[i] = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
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
  append_block<D, F16>(lo, factor, inv, codes + 8 * b0, scales + b0, held ? held + 16 * b0 : held);
  append_block<D, F16>(hi, factor, inv, codes + 8 * b1, scales + b1, held ? held + 16 * b1 : held);
}

int launch_kv4_append(const Kv4AppendArgs& a, bool f16, cudaStream_t stream) {
  const void* fn =
      a.head_dim == 64 ? (f16 ? reinterpret_cast<const void*>(lora_kv4_append_kernel<64, true>)
                              : reinterpret_cast<const void*>(lora_kv4_append_kernel<64, false>))
                       : (f16 ? reinterpret_cast<const void*>(lora_kv4_append_kernel<128, true>)
                              : reinterpret_cast<const void*>(lora_kv4_append_kernel<128, false>));
  const long long threads = static_cast<long long>(a.max_num_tokens) *
                            (a.num_q_heads + 2 * a.num_kv_heads) * (a.head_dim / 32);
  const long long grid = (threads + kAppendThreads - 1) / kAppendThreads;
  if (grid > 0x7FFFFFFFll) return -3;
  Kv4AppendArgs p = a;
  return launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(kAppendThreads), 0, stream, 0, &p);
}

}  // namespace grg
