// The 4-bit cache's layout and its number formats (sm_103a).
#pragma once

#include "common.cuh"

namespace grg {

constexpr uint32_t kStatusBadNumTokens = 0x2u;
constexpr uint32_t kStatusBadSlot = 0x10u;
constexpr uint32_t kStatusBadPosition = 0x20u;
constexpr uint32_t kStatusBadLength = 0x40u;

// A block of 16 tokens of one head: K codes, V codes, K scales, V scales.
template <int D>
struct Kv4Block {
  static constexpr int kTokens = 16;
  static constexpr int kCodeRow = D / 2;    // bytes of one token's codes
  static constexpr int kScaleRow = D / 16;  // bytes of one token's scales
  static constexpr int kK = 0;
  static constexpr int kV = 16 * kCodeRow;
  static constexpr int kKScale = 2 * kV;
  static constexpr int kVScale = kKScale + 16 * kScaleRow;
  static constexpr int kBytes = 18 * D;
};

// Four bytes of e2m1 codes (8 values, low nibble first) as four fp16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Eight floats to e2m1 codes (to the nearest, ties to even, saturating at 6).
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float* f) {
  uint32_t w;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(w)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return w;
}
// Products of two fp16 pairs (of a code and its scale: exact).
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two e4m3 bytes (low one first) as an fp16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
  return h;
}
// Two floats as e4m3 bytes (lo in the low byte), to the nearest, saturating.
__device__ __forceinline__ uint32_t f32x2_to_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
  return unpack_f16x2(e4m3x2_to_f16(b & 0xFFu)).x;
}

// |v| as an integer that orders like the number, NaN above infinity: a maximum
// over these keeps a NaN, which fmaxf drops.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

}  // namespace grg
