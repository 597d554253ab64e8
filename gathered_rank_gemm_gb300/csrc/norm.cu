// Residual addition and root-mean-square norm with 16-bit and 8-bit outputs:
//   z = x + r;  n = z * rsqrt(mean(z^2) + eps) * w;  y = 16-bit(n);
//   scale = max(max|n| / 448, 2^-100) over a row or 128 columns;  y8 = e4m3(n / scale)
// One CTA per row; the row's z is held in shared memory in fp32 between the
// sum of squares, the maximum and the stores, so x and r are read once.
#include "kv4.cuh"
#include "launch.h"
#include "layer.h"

namespace grg {

namespace {
constexpr int kNormThreads = 256;
constexpr float kMinScale = 7.888609052210118e-31f;  // 2^-100
constexpr float kInv448 = 1.0f / 448.0f;

template <bool F16>
__device__ __forceinline__ float load16(const uint16_t* p) {
  if constexpr (F16) return __half2float(*reinterpret_cast<const __half*>(p));
  return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
}
template <bool F16>
__device__ __forceinline__ uint16_t round16(float v) {
  if constexpr (F16) return __half_as_ushort(__float2half_rn(v));
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
// max(a / 448, 2^-100) of a maximum taken over abs_bits: NaN stays NaN.
__device__ __forceinline__ float scale_of(uint32_t bits) {
  const float s = __uint_as_float(bits) * kInv448;
  return s < kMinScale ? kMinScale : s;
}
}  // namespace

template <bool F16>
__global__ void __launch_bounds__(kNormThreads) lora_add_rmsnorm_kernel(const NormArgs p) {
  extern __shared__ float z[];
  __shared__ float s_sum[kNormThreads / 32];
  __shared__ uint32_t s_max[kNormThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x;
  const int raw = *p.num_tokens;
  const int n = min(max(raw, 0), p.max_num_tokens);
  if (raw != n && p.status && t == 0 && tid == 0) atomicOr(p.status, kStatusBadNumTokens);
  if (t >= n) return;
  const uint16_t* x = p.x + t * p.x_stride;
  const uint16_t* r = p.residual ? p.residual + t * p.residual_stride : nullptr;
  uint16_t* ro = p.residual_out ? p.residual_out + t * p.residual_out_stride : nullptr;
  float sum = 0.0f;
  for (int h = tid; h < p.hidden; h += kNormThreads) {
    float v = load16<F16>(x + h);
    if (r) v += load16<F16>(r + h);
    z[h] = v;
    sum += v * v;
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = 0.0f;
  for (int i = 0; i < kNormThreads / 32; ++i) sum += s_sum[i];
  const float inv = rsqrtf(sum / static_cast<float>(p.hidden) + p.eps);
  for (int h = tid; h < p.hidden; h += kNormThreads) {
    const float v = z[h];
    const float m = v * inv * load16<F16>(p.weight + h);
    z[h] = m;
    if (ro) ro[h] = round16<F16>(v);
    if (p.y) p.y[t * p.y_stride + h] = round16<F16>(m);
  }
  if (!p.y8) return;
  __syncthreads();
  uint8_t* y8 = p.y8 + t * p.y8_stride;
  if (p.group == p.hidden) {
    uint32_t top = 0;
    for (int h = tid; h < p.hidden; h += kNormThreads) top = max(top, abs_bits(z[h]));
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s_max[warp] = top;
    __syncthreads();
    for (int i = 0; i < kNormThreads / 32; ++i) top = max(top, s_max[i]);
    const float scale = scale_of(top);
    if (tid == 0) p.y8_scale[t] = scale;
    for (int h = tid; h < p.hidden; h += kNormThreads)
      y8[h] = static_cast<uint8_t>(f32x2_to_e4m3(z[h] / scale, 0.0f));
  } else {
    const int groups = p.hidden / 128;
    for (int g = warp; g < groups; g += kNormThreads / 32) {
      uint32_t top = 0;
      for (int i = lane; i < 128; i += 32) top = max(top, abs_bits(z[g * 128 + i]));
      const float scale = scale_of(__reduce_max_sync(0xffffffffu, top));
      if (lane == 0) p.y8_scale[static_cast<long long>(t) * groups + g] = scale;
      for (int i = lane; i < 128; i += 32)
        y8[g * 128 + i] = static_cast<uint8_t>(f32x2_to_e4m3(z[g * 128 + i] / scale, 0.0f));
    }
  }
}

int launch_add_rmsnorm(const NormArgs& a, bool f16, cudaStream_t stream) {
  const void* fn = f16 ? reinterpret_cast<const void*>(lora_add_rmsnorm_kernel<true>)
                       : reinterpret_cast<const void*>(lora_add_rmsnorm_kernel<false>);
  const size_t smem = static_cast<size_t>(a.hidden) * 4;
  if (ensure_smem_attr(fn, smem) != 0) return -6;
  NormArgs p = a;
  return launch_pdl(fn, dim3(a.max_num_tokens), dim3(kNormThreads), smem, stream, 0, &p);
}

}  // namespace grg
