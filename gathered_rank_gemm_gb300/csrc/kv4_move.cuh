// Moving tokens' entries (K and V, codes and scales, of one head) about in the 4-bit cache.
#pragma once

#include "kv4.cuh"

namespace grg {

// An entry is moved by D / 16 lanes: each has 16 bytes of codes (the first half of them K's,
// the other V's), lanes 0 and 1 the scales of K and V besides.
template <int D>
struct Kv4Entry {
  using B = Kv4Block<D>;
  static constexpr int kLanes = D / 16;
  using Scales = typename std::conditional<D == 128, uint2, uint32_t>::type;
  static_assert(sizeof(Scales) == B::kScaleRow, "a token's scales of K or of V");

  uint4 codes;
  Scales scales;

  // Where lane `part` of token r of a block finds its codes, and lanes 0 and 1 their scales.
  __device__ __forceinline__ static int codes_at(int r, int part) {
    constexpr int half = kLanes / 2;
    return (part < half ? B::kK : B::kV) + r * B::kCodeRow + 16 * (part % half);
  }
  __device__ __forceinline__ static int scales_at(int r, int part) {
    return (part == 0 ? B::kKScale : B::kVScale) + r * B::kScaleRow;
  }
  // (volatile: the compiler would move a load into the condition around its store, where the
  // next one then waits for it: one move 5.5 thousand cycles, now 1.5)
  __device__ __forceinline__ void load(const uint8_t* block, int r, int part) {
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(codes.x), "=r"(codes.y), "=r"(codes.z), "=r"(codes.w)
                 : "l"(block + codes_at(r, part)));
    if (part < 2) {
      if constexpr (D == 128)
        asm volatile("ld.global.v2.u32 {%0, %1}, [%2];\n" : "=r"(scales.x), "=r"(scales.y) : "l"(block + scales_at(r, part)));
      else
        asm volatile("ld.global.u32 %0, [%1];\n" : "=r"(scales) : "l"(block + scales_at(r, part)));
    }
  }
  __device__ __forceinline__ void store(uint8_t* block, int r, int part) const {
    *reinterpret_cast<uint4*>(block + codes_at(r, part)) = codes;
    if (part < 2) *reinterpret_cast<Scales*>(block + scales_at(r, part)) = scales;
  }
};

// A paged cache and one sequence's pages: the block that holds key j of head h (null: its
// page is not in the cache).
struct Kv4Pages {
  uint8_t* cache;
  const int32_t* table;
  int num_pages, num_kv_heads, page_size;

  template <int D>
  __device__ __forceinline__ uint8_t* block(int j, int h) const {
    const int pg = j / page_size;
    return block_of_page<D>(__ldg(table + pg), j - pg * page_size, h);
  }
  template <int D>
  __device__ __forceinline__ uint8_t* block_of_page(int page, int in_page, int h) const {
    if (page < 0 || page >= num_pages) return nullptr;
    return cache + ((static_cast<long long>(page) * num_kv_heads + h) * (page_size / 16) + in_page / 16) *
                       Kv4Block<D>::kBytes;
  }
};

}  // namespace grg
