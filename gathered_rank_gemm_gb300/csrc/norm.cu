// Residual addition and root-mean-square norm with 16-bit and 8-bit outputs:
//   z = x + r;  n = z * rsqrt(mean(z^2) + eps) * w;  y = 16-bit(n);
//   scale = max(max|n| / 448, 2^-100) over a row or 128 columns;  y8 = e4m3(n / scale)
// Bound by HBM (9 bytes an element with every output): one CTA per row, the row
// in registers between its one read and its one write, 16-byte accesses.  A
// scale of 128 columns is the maximum over 16 neighbouring lanes.
// Measured (GB300, bf16, 16-bit and 8-bit outputs): 8192 rows of 4096 46.2 us, 0.97 of
// the measured copy rate; 777 of 11008 (fp16) 15.8 us, 0.72: CTAs come and go in two and
// a half waves; 256 of 4096 2.9 us and one row 2.2 us, where a launch is about 2.
#include "kv4.cuh"
#include "launch.h"
#include "layer.h"

namespace grg {

namespace {
constexpr int kNormThreads = 384;      // of a CTA; more only where a row needs them
constexpr int kNormMaxThreads = 1024;
constexpr float kMinScale = 7.888609052210118e-31f;  // 2^-100
constexpr float kInv448 = 1.0f / 448.0f;
constexpr float kMaxFloat = 3.40282347e38f;
constexpr float kMaxInv = 1073741824.0f;  // 2^30: mean(z^2) + eps below 2^-60
constexpr float kUp = 1208925819614629174706176.0f, kDown = 1.0f / kUp;  // 2^80, 2^-80

// max(a / 448, 2^-100) of a maximum taken over abs_bits: NaN stays NaN.
__device__ __forceinline__ float scale_of(uint32_t bits) {
  const float s = __uint_as_float(bits) * kInv448;
  return s < kMinScale ? kMinScale : s;
}
}  // namespace

// Thread i of a CTA holds the row's chunks (of 8 columns) i, i + threads, ... , CH of them.
template <int CH, bool F16, int MAXT>
__global__ void __launch_bounds__(MAXT) lora_add_rmsnorm_kernel(const NormArgs p) {
  __shared__ float s_sum[32];
  __shared__ uint32_t s_max[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int chunks = p.hidden >> 3;
  pdl_wait();
  pdl_launch_dependents();
  const long long t = blockIdx.x;
  const int raw = *p.num_tokens;
  const int n = min(max(raw, 0), p.max_num_tokens);
  if (raw != n && p.status && t == 0 && tid == 0) atomicOr(p.status, kStatusBadNumTokens);
  if (t >= n) return;
  const uint4* x = reinterpret_cast<const uint4*>(p.x + t * p.x_stride);
  const uint4* r = p.residual ? reinterpret_cast<const uint4*>(p.residual + t * p.residual_stride) : nullptr;
  const uint4* w = reinterpret_cast<const uint4*>(p.weight);
  uint4 xv[CH], rv[CH], wv[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * blockDim.x;
    const bool in = c < chunks;
    xv[i] = in ? __ldcs(x + c) : make_uint4(0, 0, 0, 0);
    rv[i] = in && r ? __ldcs(r + c) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * blockDim.x;
    wv[i] = c < chunks ? __ldg(w + c) : make_uint4(0, 0, 0, 0);
  }
  float z[CH][8], sum = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const uint32_t a[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
    const uint32_t b[4] = {rv[i].x, rv[i].y, rv[i].z, rv[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack_t<F16>(a[e]), g = unpack_t<F16>(b[e]);
      z[i][2 * e] = r ? f.x + g.x : f.x;
      z[i][2 * e + 1] = r ? f.y + g.y : f.y;
      sum += z[i][2 * e] * z[i][2 * e] + z[i][2 * e + 1] * z[i][2 * e + 1];
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  if (p.residual_out) {
    uint4* ro = reinterpret_cast<uint4*>(p.residual_out + t * p.residual_out_stride);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * blockDim.x;
      if (c < chunks)
        ro[c] = make_uint4(pack_t<F16>(z[i][0], z[i][1]), pack_t<F16>(z[i][2], z[i][3]),
                           pack_t<F16>(z[i][4], z[i][5]), pack_t<F16>(z[i][6], z[i][7]));
    }
  }
  __syncthreads();
  sum = lane < warps ? s_sum[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  float inv = rsqrtf(sum / static_cast<float>(p.hidden) + p.eps);
  if (sum > kMaxFloat || inv > kMaxInv) {
    // rare: squares that leave the range, whose mean does not leave its root's.  The row
    // is scaled by a power of two and summed again (the whole CTA comes here).
    const float f = sum > kMaxFloat ? kDown : kUp;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        z[i][e] *= f;
        sum += z[i][e] * z[i][e];
      }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    sum = lane < warps ? s_sum[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    inv = rsqrtf(sum / static_cast<float>(p.hidden) + p.eps * f * f);
  }
  uint32_t top = 0, tops[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const uint32_t b[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w};
    tops[i] = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 g = unpack_t<F16>(b[e]);
      z[i][2 * e] *= inv * g.x;
      z[i][2 * e + 1] *= inv * g.y;
      tops[i] = max(tops[i], max(abs_bits(z[i][2 * e]), abs_bits(z[i][2 * e + 1])));
    }
    if (tid + i * blockDim.x >= chunks) tops[i] = 0;  // 0 * inv may be a NaN
    top = max(top, tops[i]);
  }
  if (p.y) {
    uint4* y = reinterpret_cast<uint4*>(p.y + t * p.y_stride);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * blockDim.x;
      if (c < chunks)
        y[c] = make_uint4(pack_t<F16>(z[i][0], z[i][1]), pack_t<F16>(z[i][2], z[i][3]),
                          pack_t<F16>(z[i][4], z[i][5]), pack_t<F16>(z[i][6], z[i][7]));
    }
  }
  if (!p.y8) return;
  float down[CH], scale[CH];  // a scale's reciprocal, and the scale where it is finite
  auto use = [&](int i, float s) {
    down[i] = __frcp_rn(s);
    scale[i] = s > kMaxFloat ? 0.0f : s;
  };
  if (p.group == p.hidden) {
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s_max[warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, lane < warps ? s_max[lane] : 0u);
    const float s = scale_of(top);
    if (tid == 0) p.y8_scale[t] = s;
    use(0, s);
#pragma unroll
    for (int i = 1; i < CH; ++i) down[i] = down[0], scale[i] = scale[0];
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
#pragma unroll
      for (int o = 8; o; o >>= 1) tops[i] = max(tops[i], __shfl_xor_sync(0xffffffffu, tops[i], o));
      const float s = scale_of(tops[i]);
      const int c = tid + i * blockDim.x;
      if (c < chunks && (lane & 15) == 0) p.y8_scale[t * (chunks >> 4) + (c >> 4)] = s;
      use(i, s);
    }
  }
  uint2* y8 = reinterpret_cast<uint2*>(p.y8 + t * p.y8_stride);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * blockDim.x;
    // n / scale rounded once (Markstein, 1990): with the correctly rounded reciprocal r,
    // q - (q scale - n) r is the quotient's nearest; in this order of the signs -0 stays -0.
    // (An infinite scale leaves q as it is.)
    auto over = [&](float n) {
      const float q = __fmul_rn(n, down[i]);
      return __fmaf_rn(-__fmaf_rn(q, scale[i], -n), down[i], q);
    };
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = f32x2_to_e4m3(over(z[i][2 * e]), over(z[i][2 * e + 1]));
    if (c < chunks) y8[c] = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
  }
}

namespace {
template <int CH, int MAXT>
int run_norm(const NormArgs& a, bool f16, cudaStream_t stream) {
  const void* fn = f16 ? reinterpret_cast<const void*>(lora_add_rmsnorm_kernel<CH, true, MAXT>)
                       : reinterpret_cast<const void*>(lora_add_rmsnorm_kernel<CH, false, MAXT>);
  const int chunks = a.hidden / 8;
  const int threads = ((chunks + CH - 1) / CH + 31) / 32 * 32;
  NormArgs p = a;
  return launch_pdl(fn, dim3(a.max_num_tokens), dim3(threads), 0, stream, 0, &p);
}
}  // namespace

// Chunks a thread holds: few for short rows, whose CTAs would else be small (one row
// of 4096: 2.2 us with two, 2.4 us with four; 2048 of 5120: 16.8 and 17.6 us), four
// where two would take more than kNormThreads (4096 of 8192: 48.0 us with
// four, 52.8 us with two; 777 of 11008: 15.8 and 19.0 us).
int launch_add_rmsnorm(const NormArgs& a, bool f16, cudaStream_t stream) {
  const int chunks = a.hidden / 8;
  if (chunks <= 256) return run_norm<1, kNormThreads>(a, f16, stream);
  if (chunks <= 2 * kNormThreads) return run_norm<2, kNormThreads>(a, f16, stream);
  if (chunks <= 4 * kNormThreads) return run_norm<4, kNormThreads>(a, f16, stream);
  return run_norm<4, kNormMaxThreads>(a, f16, stream);
}

}  // namespace grg
