// What the two attention kernels over the 4-bit cache share (internal): a
// sequence's rows and keys, and which of the two kernels takes it.
#pragma once

#include "kv4.cuh"
#include "layer.h"

namespace grg {

// One sequence's rows and keys, clamped to what the buffers hold.
struct Kv4Seq {
  int q0;    // first row
  int rows;  // rows (the last one stands at position kv - 1)
  int take;  // rows that get an output: the first max_q_len
  int kv;    // keys
  bool odd;  // something had to be clamped
  __device__ __forceinline__ static Kv4Seq of(const Kv4AttnArgs& p, int b) {
    const int a = p.q_start[b], e = p.q_start[b + 1], k = p.kv_len[b];
    Kv4Seq s;
    s.q0 = min(max(a, 0), p.max_num_tokens);
    s.rows = min(max(e, s.q0), p.max_num_tokens) - s.q0;
    s.take = min(s.rows, p.max_q_len);
    s.kv = static_cast<int>(min(static_cast<long long>(max(k, 0)), p.table_stride * p.page_size));
    s.odd = a != s.q0 || e != s.q0 + s.rows || s.kv != k || s.take != s.rows;
    return s;
  }
  // The position of row i, and the first key that a row there sees.
  __device__ __forceinline__ int pos(int i) const { return kv - rows + i; }
  __device__ __forceinline__ int first_key(int i, int window) const {
    const int at = pos(i);  // (below 0 for a row without keys: at - window may not fit 32 bits)
    return window > 0 && at >= window ? at - window + 1 : 0;
  }

  // Whether the decode kernel takes the sequence: few packed rows, or a short tree.
  template <bool TREE>
  __device__ __forceinline__ bool few(const Kv4AttnArgs& a, int group, int max_packed_rows) const {
    const long long packed = static_cast<long long>(take) * group;
    return packed <= max_packed_rows || (TREE && packed <= a.short_rows && kv <= a.short_keys);
  }

  // Which keys rows see.  A row of a sequence sees a run of keys that ends at its own
  // position; a row of a tree (TREE) those in front of all rows' own, from its window's
  // first on, and of the rows' own what its mask names.
  __device__ __forceinline__ int before() const { return kv - rows; }
  // The last key of row i's run.
  template <bool TREE>
  __device__ __forceinline__ int run_last(int i) const {
    return TREE ? before() - 1 : pos(i);
  }
  // The first.  A row of a tree stands as far behind the keys in front as it has ancestors.
  template <bool TREE>
  __device__ __forceinline__ int run_first(const Kv4AttnArgs& a, int i) const {
    if constexpr (!TREE) return first_key(i, a.window);
    if (a.window == 0) return 0;
    const uint32_t* mask = a.tree_mask + static_cast<long long>(q0 + i) * a.tree_words;
    int named = 0;
    for (int w = 0; w < a.tree_words && 32 * w < rows; ++w)
      named += __popc(mask[w] & (rows - 32 * w >= 32 ? ~0u : (1u << (rows - 32 * w)) - 1u));
    return first_key(max(named - 1, 0), a.window);
  }
  // Bounds for the rows i0 .. i1: no row sees a key in front of keys_first or from keys_end
  // on, and every row's run reaches from run_first_max to run_last(i0).
  template <bool TREE>
  __device__ __forceinline__ int keys_first(int i0, int window) const {
    return first_key(TREE ? 0 : i0, window);
  }
  template <bool TREE>
  __device__ __forceinline__ int keys_end(int i1) const {
    return TREE ? kv : pos(i1) + 1;
  }
  template <bool TREE>
  __device__ __forceinline__ int run_first_max(int i1, int window) const {
    return first_key(TREE ? rows - 1 : i1, window);
  }
};

// The lowest n bits (none below 0, all from 32 on), and all but those.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// Of 32 keys from key0 on, those that a row of a tree sees, as bits: the run [lo, before) and
// what the row's mask names among the rows' own keys [before, kv).
__device__ __forceinline__ uint32_t tree_sees(const Kv4AttnArgs& a, const Kv4Seq& s, long long row, int lo,
                                              int key0) {
  const int c0 = key0 - s.before();  // the first key among the rows' own, rounded down to a word
  const int w0 = c0 >> 5;
  uint32_t bits = low_bits(-c0) & ~low_bits(lo - key0);
  if (c0 > -32) {
    const uint32_t* mask = a.tree_mask + row * a.tree_words;
    const uint32_t x = w0 >= 0 && w0 < a.tree_words ? __ldg(mask + w0) : 0u;
    const uint32_t y = w0 + 1 < a.tree_words ? __ldg(mask + w0 + 1) : 0u;  // (w0 + 1 >= 0)
    bits |= __funnelshift_r(x, y, c0 & 31) & ~low_bits(-c0);
  }
  return bits & low_bits(s.kv - key0);
}

// a / b of values that are rarely past 32 bits (a >= 0, b > 0); a 64-bit division takes
// some hundred cycles on every call's way.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b))
                              : a / b;
}

// The last of the 32 * PER ascending values that is not above x (values[0] is not), by
// a whole warp in two looks.
template <int PER>
__device__ __forceinline__ int last_not_past(const long long* values, long long x, int lane) {
  static_assert(PER <= 32, "the second look is one value a lane");
  const int block = __popc(__ballot_sync(0xffffffffu, values[lane * PER] <= x)) - 1;
  const bool in = lane < PER && values[block * PER + min(lane, PER - 1)] <= x;
  return block * PER + __popc(__ballot_sync(0xffffffffu, in)) - 1;
}

// 2^x.
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}

// The power of two that takes a row whose largest magnitude is `top` into
// [2^14, 2^15), where fp16 holds its 16-bit elements without loss, and its
// inverse; 1 for a row of zeros (or of no finite maximum).
__device__ __forceinline__ void row_factor(float top, float& up, float& down) {
  int e = static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127;
  e = (top == 0.0f || e > 127) ? 14 : max(e, -112);
  up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
  down = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
}

// What turns a row's products into scores in units of log2: its factor's inverse times the
// call's.  Kept among the normal numbers, whose ends leave scores of 0 and beyond fp32
// either way: 0 times a masked key's -infinity, or infinity times 0, would be a NaN.
__device__ __forceinline__ float score_factor(float down, float scale) {
  return fminf(fmaxf(down * scale, 1.17549435e-38f), 3.40282347e38f);
}

}  // namespace grg
