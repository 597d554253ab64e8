// What the kernels of the key weights share (internal): a sequence's rows and keys.
#pragma once

#include "kv4_attention.cuh"
#include "kv4_move.cuh"

namespace grg {

// One sequence's rows (its own, or those of its path) and keys, clamped to what the buffers hold.
struct WeightSeq {
  int q0;      // its first row in q
  int q_rows;  // rows that it has there
  int rows;    // rows that count, the last of them at position kv - 1
  int take;    // those that are summed: the first max_q_len
  int kv;      // keys
  int end;     // keys that have a weight to go to
  bool odd;    // something had to be clamped
  __device__ __forceinline__ static WeightSeq of(const Kv4WeightsArgs& p, int b) {
    const int a = p.q_start[b], e = p.q_start[b + 1], k = p.kv_len[b];
    WeightSeq s;
    s.q0 = min(max(a, 0), p.max_num_tokens);
    s.q_rows = min(max(e, s.q0), p.max_num_tokens) - s.q0;
    s.odd = a != s.q0 || e != s.q0 + s.q_rows;
    s.rows = s.q_rows;
    if (p.path) {
      const int len = p.path_len[b];
      s.rows = min(max(len, 0), min(s.q_rows, p.max_path));
      s.odd = s.odd || s.rows != len;
    }
    s.take = min(s.rows, p.max_q_len);
    s.kv = static_cast<int>(min(static_cast<long long>(max(k, 0)), p.table_stride * p.page_size));
    s.end = min(s.kv, p.capacity);
    s.odd = s.odd || s.kv != k || s.take != s.rows || s.end != s.kv;
    return s;
  }
  __device__ __forceinline__ int pos(int i) const { return kv - rows + i; }
  // The first key in row i's window.  A path's row sees all of its ancestors besides, as the tree's
  // attention had it: the window hides keys in front of the path only.  (The first row has none.)
  __device__ __forceinline__ int first_key(int i, int window) const {
    const int at = pos(i);
    return window > 0 && at >= window ? at - window + 1 : 0;
  }
  // Blocks of 16 keys that some row sees or that are the rows' own: [first, first + count).
  __device__ __forceinline__ int first_block(int window) const { return first_key(0, window) / 16; }
  __device__ __forceinline__ int blocks(int window) const {
    return rows > 0 ? max((end + 15) / 16 - first_block(window), 0) : 0;
  }
  // Row i's place in q; below 0: the path names none.
  __device__ __forceinline__ int row_in_q(const Kv4WeightsArgs& p, int b, int i) const {
    if (!p.path) return q0 + i;
    const int c = __ldg(p.path + static_cast<long long>(b) * p.max_path + i);
    return c < 0 || c >= q_rows ? -1 : q0 + c;
  }
};

// Sequences with more than max_packed_rows rows x heads of a key head (kv4_weights_tc.cu).
int launch_kv4_weights_tc(const Kv4WeightsArgs& a, int max_packed_rows, bool f16, cudaStream_t stream);

}  // namespace grg
