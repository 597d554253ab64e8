/*
 * gathered_rank_gemm — multi-LoRA shrink / expand over an unsorted,
 * mixed-adapter token batch, for NVIDIA GB300 (sm_103a).
 *
 * The operation (one LoRA-wrapped linear layer):
 *
 *   "[V1] LoRA - Add triton kernels for V1" (vLLM PR 13096), section "Why do
 *   we need a new set of kernels": the batch is NOT sorted by LoRA id; the
 *   kernels are given the token -> LoRA map and use it to load each token's
 *   rows, then run the low-rank (SGMV-style) matmuls.  Point 1 of "Kernel Code
 *   Change": the launch grid must not depend on the batch, so the calls can be
 *   captured once in a CUDA graph.
 *   "[Kernel] LoRA - Enable CUDAGraphs for V1" (vLLM PR 14626): buffers are
 *   static, sized by max_num_tokens, and the pad rows past the valid tokens are
 *   not zeroed, so they must never be read into an output.
 *
 * With m = token_lora_mapping (-1 = no adapter), n valid tokens, L adapter
 * slots, rank R and S in {1,2,3} output slices of widths N_s at column
 * offsets off_s = N_0 + ... + N_{s-1}:
 *
 *   lora_prepare_metadata: stable grouping of t in [0, n) by m[t]
 *   lora_shrink:  u[s][t][r] = scale * sum_h x[t][h] * A_s[m[t]][r][h]   (fp32 out)
 *   lora_expand:  y[t][off_s + j] = bf16( y[t][off_s + j]
 *                                       + sum_r u[s][t][r] * B_s[m[t]][r][j] )
 *
 * for t < n with 0 <= m[t] < L.  Rows of tokens with m[t] = -1 and rows t >= n
 * are never read from x and never read from or written to u and y.
 *
 * Conventions for every call:
 *  - Every array argument is a DEVICE pointer owned by the caller, except the
 *    small per-slice arrays (lora_a, lora_b, slice_width), which are HOST
 *    arrays of num_slices entries read during the call (their device pointers
 *    are copied into the kernel parameters).  The library never allocates,
 *    frees or synchronises (lora_read_status excepted).
 *  - bf16 data is passed as uint16_t bit patterns (IEEE bfloat16).
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) on the current device, so every call can be captured into a CUDA
 *    graph.  The number of valid tokens n lives in device memory, so one
 *    captured graph serves every n <= max_num_tokens.
 *  - Kernels are launched with programmatic dependent launch enabled, so a
 *    kernel may start while the one ahead of it on the stream is finishing.
 *    Before its dependency wait (which returns once every earlier kernel on
 *    the stream has completed and its writes are visible) a kernel of this
 *    library only
 *      - reads the tile records in the workspace, which only
 *        lora_prepare_metadata writes and which it makes visible before it
 *        lets the next kernel start (so nothing else may write the workspace
 *        while calls that use it are in flight), and
 *      - prefetches weights and activation rows into L2, which is the GPU's
 *        coherence point: a prefetch never yields stale data.
 *    Every copy into shared memory and every other read comes after the
 *    wait, with one exception inside lora_shrink_expand (and its fp16 and
 *    paged forms): its second kernel loads B and its y rows before the wait,
 *    because the kernel ahead of it is the same call's shrink, which writes
 *    neither and lets the second kernel start only after its own wait.  So
 *    any kernel may come right before any call, including one that rewrites
 *    the weights, x or y.  A kernel whose CTAs have no work still waits
 *    before it exits, so stream order holds through it.
 *  - Return value: LORA_OK when the work was enqueued, a negative LORA_ERR_*
 *    code when an argument was rejected (nothing is launched) or the launch
 *    failed.  Problems that only the data reveals (a LoRA id outside [-1, L),
 *    n outside [0, max_num_tokens]) cannot be reported synchronously: they set
 *    bits in the status word inside the workspace (lora_read_status), and the
 *    offending tokens are treated as having no adapter / n is clamped.
 */
#ifndef GATHERED_RANK_GEMM_H
#define GATHERED_RANK_GEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_OK 0
#define LORA_ERR_NULL (-1)       /* a required pointer is NULL */
#define LORA_ERR_ALIGN (-2)      /* a pointer or row stride breaks the 16-byte rule */
#define LORA_ERR_SHAPE (-3)      /* a size is outside the supported set */
#define LORA_ERR_WORKSPACE (-4)  /* workspace too small */
#define LORA_ERR_LAUNCH (-5)     /* the CUDA launch failed (cudaGetLastError) */
#define LORA_ERR_CUDA (-6)       /* another CUDA runtime call failed */

#define LORA_STATUS_BAD_LORA_ID 0x1u     /* some m[t], t < n, was outside [-1, L) */
#define LORA_STATUS_BAD_NUM_TOKENS 0x2u  /* n was outside [0, max_num_tokens]; clamped */
#define LORA_STATUS_TIMEOUT 0x4u         /* a kernel's bounded wait for its own copies gave up;
                                            the outputs of that call are unspecified */
#define LORA_STATUS_BAD_WEIGHT 0x8u      /* a paged weight address was not 16-byte aligned */
#define LORA_STATUS_BAD_SLOT 0x10u       /* a cache slot or page id lay outside the cache */
#define LORA_STATUS_BAD_POSITION 0x20u   /* a token's position lay outside the rotation table */
#define LORA_STATUS_BAD_LENGTH 0x40u     /* a sequence's rows or keys did not fit their buffers */

#define LORA_MAX_SLICES 3
#define LORA_MAX_LORAS 1024
#define LORA_MAX_NUM_TOKENS (1 << 22)

/*
 * Bytes of device workspace that lora_prepare_metadata fills and lora_shrink /
 * lora_expand read: a status word, the clamped n and, for tile heights of
 * 16, 32, 64 and 128 tokens, the list of tile records (adapter, count and the
 * tile's token ids) that the fixed-grid kernels walk.  About 4 * 4 bytes per
 * token plus 1 KB per adapter (277 KB at 8192 tokens and 128 LoRAs).  Returns
 * 0 for sizes outside the supported range.  Besides the grouping kernel, the
 * shrink and expand kernels may OR LORA_STATUS_TIMEOUT into its status word.
 */
size_t lora_workspace_size(int64_t max_num_tokens, int64_t max_loras);

/*
 * Stable grouping of the batch's tokens by LoRA id ("[V1] LoRA - Add triton
 * kernels for V1", "Why do we need a new set of kernels": V1 keeps the batch
 * unsorted, so the grouping is computed on the device from the token -> LoRA
 * map; "[Kernel] LoRA - Enable CUDAGraphs for V1": the map is a static
 * max_num_tokens buffer).  A histogram / prefix-sum / stable scatter, run by
 * one CTA when max_num_tokens <= 1024 and max_loras <= 128 (one token per
 * thread), else by one thread-block cluster (one CTA per 1024 tokens of
 * max_num_tokens, up to 8); the grid depends only on max_num_tokens and
 * max_loras, not on the data.
 *
 *   token_lora_mapping   int32[max_num_tokens]; entries t >= n may be loaded
 *                        (the one-CTA kernel loads every entry at once with
 *                        n) but never affect any output
 *   num_tokens           device int32: n
 *   sorted_token_ids     int32[max_num_tokens] out: tokens of LoRA 0 in
 *                        ascending order, then LoRA 1, ..., then the tokens
 *                        without an adapter; entries n.. are -1
 *   num_tokens_per_lora  int32[max_loras + 1] out: entry L counts tokens
 *                        without an adapter
 *   lora_token_start_loc int32[max_loras + 2] out: exclusive prefix sum of the
 *                        counts; entry L+1 equals n
 *   workspace            lora_workspace_size(max_num_tokens, max_loras) bytes,
 *                        16-byte aligned; its status word is OR-ed (never
 *                        cleared here) and the rest is overwritten
 * Sizes: 1 <= max_num_tokens <= LORA_MAX_NUM_TOKENS, 1 <= max_loras <= LORA_MAX_LORAS.
 */
int lora_prepare_metadata(const int32_t *token_lora_mapping, const int32_t *num_tokens,
                          int64_t max_num_tokens, int64_t max_loras,
                          int32_t *sorted_token_ids, int32_t *num_tokens_per_lora,
                          int32_t *lora_token_start_loc, void *workspace,
                          size_t workspace_bytes, void *stream);

/*
 * Shrink ("[V1] LoRA - Add triton kernels for V1": gather each token's input
 * row through the token -> LoRA information and multiply by its adapter's A):
 *   u[s][t][r] = c(m[t]) * sum_h x[t][h] * A_s[m[t]][r][h]  (bf16 in, fp32 out)
 *   c(l) = scale, or scale * lora_scales[l] (in fp32) when lora_scales is given
 *
 *   x                bf16[max_num_tokens][x_row_stride], hidden columns used
 *   lora_a           HOST array of num_slices device pointers, each
 *                    bf16[max_loras][rank][hidden] row-major
 *   lora_scales      NULL, or device fp32[max_loras]: a per-adapter factor on
 *                    scale (the pages are silent on per-LoRA scales)
 *   u                fp32[num_slices][max_num_tokens][rank] out; only rows of
 *                    adapter tokens t < n are written
 *   sorted_token_ids, lora_token_start_loc, workspace: from lora_prepare_metadata
 *                    with the same max_num_tokens / max_loras
 * Sizes: hidden a multiple of 8, rank in {8, 16, 32, 64, 128}, 1 <= num_slices
 * <= 3; x, every A_s and u 16-byte aligned, x_row_stride a multiple of 8 and
 * >= hidden.  Accumulation is fp32 (tensor cores, bf16 operands).
 */
int lora_shrink(const uint16_t *x, int64_t x_row_stride, int64_t hidden,
                const uint16_t *const *lora_a, int num_slices, int rank, float scale,
                const float *lora_scales, float *u, const int32_t *sorted_token_ids,
                const int32_t *lora_token_start_loc,
                int64_t max_num_tokens, int64_t max_loras, const void *workspace,
                size_t workspace_bytes, void *stream);

/*
 * Expand ("[V1] LoRA - Add triton kernels for V1": same token loading, rank ->
 * width matmul added into the layer's output):
 *   y[t][off_s + j] = bf16( float(y[t][off_s + j]) + sum_r u[s][t][r] * B_s[m[t]][r][j] )
 * one round-to-nearest-even per element; y is updated in place.
 *
 *   u                fp32[num_slices][max_num_tokens][rank] (from lora_shrink)
 *   lora_b           HOST array of num_slices device pointers, each
 *                    bf16[max_loras][rank][slice_width[s]] row-major
 *   slice_width      HOST array of num_slices widths, each a multiple of 8
 *   y                bf16[max_num_tokens][y_row_stride] in/out; slice s covers
 *                    columns off_s .. off_s + slice_width[s] - 1
 *   sorted_token_ids, lora_token_start_loc, workspace: from lora_prepare_metadata
 * Sizes: y_row_stride a multiple of 8 and >= the sum of the widths; rank in
 * {8, 16, 32, 64, 128}; u, y and every B_s 16-byte aligned.  The rank
 * contraction runs on tensor cores with u split into two bf16 terms
 * (high + low part), so u keeps about 16 significant bits.
 */
int lora_expand(const float *u, const uint16_t *const *lora_b, const int64_t *slice_width,
                int num_slices, int rank, uint16_t *y, int64_t y_row_stride,
                const int32_t *sorted_token_ids, const int32_t *lora_token_start_loc,
                int64_t max_num_tokens, int64_t max_loras, const void *workspace,
                size_t workspace_bytes, void *stream);

/*
 * Shrink then expand for one layer in one call: the same arguments, results
 * and rules as lora_shrink followed by lora_expand (u is written too).  When
 * the batch is small enough for a thread-block cluster to hold a tile's whole
 * problem on chip (decode-sized batches: up to 16 k-blocks of 64 columns and
 * 48 output units of 64 columns per CTA) and every tile's cluster fits in one
 * wave, one fused kernel does both steps and the expand reads u from shared
 * memory.  Otherwise, with a workspace of at least
 * lora_shrink_expand_workspace_size bytes and a batch of up to 1024 tokens
 * with rank <= 32, the split-K path runs: the shrink's CTAs (up to 16 per
 * tile, no cluster) write partial tiles of u into the workspace and the
 * expand adds them up in CTA order (u and y then match the two separate calls
 * up to the order of the fp32 partial sums).  Else the kernels of
 * lora_shrink and lora_expand run unchanged.  Either way the work stays on
 * the GPU; lora_shrink_expand_path tells which path a shape takes.  The
 * split-K path keeps its partial tiles in the workspace: order calls that
 * share a workspace on one stream.
 */
int lora_shrink_expand(const uint16_t *x, int64_t x_row_stride, int64_t hidden,
                       const uint16_t *const *lora_a, const uint16_t *const *lora_b,
                       const int64_t *slice_width, int num_slices, int rank, float scale,
                       const float *lora_scales, float *u, uint16_t *y, int64_t y_row_stride,
                       const int32_t *sorted_token_ids, const int32_t *lora_token_start_loc,
                       int64_t max_num_tokens, int64_t max_loras, const void *workspace,
                       size_t workspace_bytes, void *stream);

/*
 * Workspace bytes that let lora_shrink_expand take its split-K path for this
 * shape: lora_workspace_size plus P * 16 * num_slices * rank * 4 bytes of
 * partial tiles per 16-token tile of the batch (P = 16 for rank <= 16, 8 for
 * rank 32: the largest split) when max_num_tokens <= 1024 and rank <= 32
 * (else just lora_workspace_size); 0 for sizes the calls reject.
 * A smaller workspace (at least lora_workspace_size) is still valid for
 * every call.
 */
size_t lora_shrink_expand_workspace_size(int64_t max_num_tokens, int64_t max_loras,
                                         int64_t hidden, const int64_t *slice_width,
                                         int num_slices, int rank);

/*
 * fp16 variants (the pages fix no input precision; models served in fp16
 * need them): the same arguments, results and rules as lora_shrink,
 * lora_expand, lora_shrink_expand, lora_shrink_partials and
 * lora_expand_partials (stacked weights), with x, A_s, B_s and y holding IEEE
 * fp16 words instead of bf16.  Accumulation stays fp32; u enters the
 * expand's tensor cores as an fp16 high part plus an fp16 residual, so |u|
 * must stay below the fp16 range (65504); y is rounded once to fp16 (round
 * to nearest even).  Paged weights and lora_apply_noalloc are bf16 only.
 */
int lora_shrink_f16(const uint16_t *x, int64_t x_row_stride, int64_t hidden,
                    const uint16_t *const *lora_a, int num_slices, int rank, float scale,
                    const float *lora_scales, float *u, const int32_t *sorted_token_ids,
                    const int32_t *lora_token_start_loc, int64_t max_num_tokens,
                    int64_t max_loras, const void *workspace, size_t workspace_bytes,
                    void *stream);
int lora_expand_f16(const float *u, const uint16_t *const *lora_b, const int64_t *slice_width,
                    int num_slices, int rank, uint16_t *y, int64_t y_row_stride,
                    const int32_t *sorted_token_ids, const int32_t *lora_token_start_loc,
                    int64_t max_num_tokens, int64_t max_loras, const void *workspace,
                    size_t workspace_bytes, void *stream);
int lora_shrink_expand_f16(const uint16_t *x, int64_t x_row_stride, int64_t hidden,
                           const uint16_t *const *lora_a, const uint16_t *const *lora_b,
                           const int64_t *slice_width, int num_slices, int rank, float scale,
                           const float *lora_scales, float *u, uint16_t *y, int64_t y_row_stride,
                           const int32_t *sorted_token_ids, const int32_t *lora_token_start_loc,
                           int64_t max_num_tokens, int64_t max_loras, const void *workspace,
                           size_t workspace_bytes, void *stream);
int lora_shrink_partials_f16(const uint16_t *x, int64_t x_row_stride, int64_t hidden,
                             const uint16_t *const *lora_a, int num_slices, int rank,
                             const int32_t *sorted_token_ids, const int32_t *lora_token_start_loc,
                             int64_t max_num_tokens, int64_t max_loras, void *workspace,
                             size_t workspace_bytes, void *stream);
int lora_expand_partials_f16(int64_t hidden, const uint16_t *const *lora_b,
                             const int64_t *slice_width, int num_slices, int rank, float scale,
                             const float *lora_scales, float *u, uint16_t *y,
                             int64_t y_row_stride, const int32_t *sorted_token_ids,
                             const int32_t *lora_token_start_loc, int64_t max_num_tokens,
                             int64_t max_loras, const void *workspace, size_t workspace_bytes,
                             void *stream);

/*
 * Paged adapter weights (the S-LoRA idea of the pages' "[Tracking] Multi-LoRA
 * Serving" overview: adapters live in separately allocated pages rather than
 * one stacked tensor).  Same arguments, results and rules as lora_shrink,
 * lora_expand and lora_shrink_expand, except that each slice's weights come
 * as a table instead of a stacked tensor:
 *   lora_a_tables   HOST array of num_slices device pointers, each to
 *                   uint64[max_loras]: the device address of adapter l's
 *                   A_s[l], bf16[rank][hidden] row-major
 *   lora_b_tables   the same for B_s[l], bf16[rank][slice_width[s]]
 * Table pointers must be 8-byte aligned.  An entry must be 16-byte aligned
 * or 0; 0 reads as an all-zero adapter (its tokens get u = 0, y unchanged),
 * and a misaligned entry reads the same way and sets LORA_STATUS_BAD_WEIGHT.
 * The tables and the weights they point to are read after the kernels'
 * dependency wait, like stacked weights.  The weights move by 16-byte cp.async
 * instead of TMA tensor maps; the one-call entry point never takes the
 * fused kernel.
 */
int lora_shrink_paged(const uint16_t *x, int64_t x_row_stride, int64_t hidden,
                      const uint64_t *const *lora_a_tables, int num_slices, int rank,
                      float scale, const float *lora_scales, float *u,
                      const int32_t *sorted_token_ids, const int32_t *lora_token_start_loc,
                      int64_t max_num_tokens, int64_t max_loras, const void *workspace,
                      size_t workspace_bytes, void *stream);
int lora_expand_paged(const float *u, const uint64_t *const *lora_b_tables,
                      const int64_t *slice_width, int num_slices, int rank, uint16_t *y,
                      int64_t y_row_stride, const int32_t *sorted_token_ids,
                      const int32_t *lora_token_start_loc, int64_t max_num_tokens,
                      int64_t max_loras, const void *workspace, size_t workspace_bytes,
                      void *stream);
int lora_shrink_expand_paged(const uint16_t *x, int64_t x_row_stride, int64_t hidden,
                             const uint64_t *const *lora_a_tables,
                             const uint64_t *const *lora_b_tables, const int64_t *slice_width,
                             int num_slices, int rank, float scale, const float *lora_scales,
                             float *u, uint16_t *y, int64_t y_row_stride,
                             const int32_t *sorted_token_ids, const int32_t *lora_token_start_loc,
                             int64_t max_num_tokens, int64_t max_loras, const void *workspace,
                             size_t workspace_bytes, void *stream);

/*
 * The two halves of lora_shrink_expand's split-K path, for callers that want
 * to place other work between them (and for timing each kernel).  Same
 * arguments and rules as lora_shrink / lora_expand, with these differences:
 *   - the shape must have max_num_tokens <= 1024 and rank <= 32, and the
 *     workspace must hold lora_shrink_expand_workspace_size bytes
 *     (LORA_ERR_SHAPE / LORA_ERR_WORKSPACE otherwise);
 *   - lora_shrink_partials splits each 16-token tile's hidden dimension over
 *     up to P CTAs (as for the workspace size above; no cluster) and writes
 *     each CTA's fp32 partial tile (its warps summed) into the workspace
 *     behind the metadata: [tile][split][16][num_slices * rank].  It does not
 *     scale and does not write u.
 *   - lora_expand_partials takes `hidden` (it fixes the split), `scale` and
 *     `lora_scales`, sums each tile's partials in CTA order, multiplies by
 *     c(lora) as lora_shrink does, writes the result to u (rows of tokens
 *     with an adapter) and adds u * B into y.
 * Run back to back on one stream they give the u and y of lora_shrink
 * followed by lora_expand up to the order of the fp32 partial sums (bit for
 * bit when the split equals lora_shrink's cluster size).  The partials of one
 * call pair live in
 * the workspace: a second pair on the same workspace must be ordered after
 * the first expand (same stream, or an event).
 */
int lora_shrink_partials(const uint16_t *x, int64_t x_row_stride, int64_t hidden,
                         const uint16_t *const *lora_a, int num_slices, int rank,
                         const int32_t *sorted_token_ids, const int32_t *lora_token_start_loc,
                         int64_t max_num_tokens, int64_t max_loras, void *workspace,
                         size_t workspace_bytes, void *stream);
int lora_expand_partials(int64_t hidden, const uint16_t *const *lora_b,
                         const int64_t *slice_width, int num_slices, int rank, float scale,
                         const float *lora_scales, float *u, uint16_t *y, int64_t y_row_stride,
                         const int32_t *sorted_token_ids, const int32_t *lora_token_start_loc,
                         int64_t max_num_tokens, int64_t max_loras, const void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * Whether one lora_shrink_expand call for this shape on the current device
 * runs the fused kernel: 1 (it does) or 2 (it does not: the split-K or the
 * two-kernel path, see lora_shrink_expand_path); a negative LORA_ERR_* code
 * for sizes the calls reject.  Host-only, no GPU work.
 */
int lora_shrink_expand_kernels(int64_t max_num_tokens, int64_t max_loras, int64_t hidden,
                               const int64_t *slice_width, int num_slices, int rank);

/*
 * Which kernels one lora_shrink_expand call (fp16 != 0: lora_shrink_expand_f16;
 * paged != 0: lora_shrink_expand_paged) runs for this shape, workspace size
 * and the current device; host-only, no GPU work:
 *   LORA_PATH_FUSED        one kernel holding a tile's whole problem on chip
 *                          (tiny batches; never with paged weights)
 *   LORA_PATH_SPLIT_PAIR   the split-K shrink, then the partial-sum expand
 *                          (needs lora_shrink_expand_workspace_size bytes)
 *   LORA_PATH_PAIR         the kernels of lora_shrink, then of lora_expand
 * A negative LORA_ERR_* code for sizes the calls reject.
 */
#define LORA_PATH_FUSED 1
#define LORA_PATH_SPLIT_PAIR 3
#define LORA_PATH_PAIR 4
int lora_shrink_expand_path(int64_t max_num_tokens, int64_t max_loras, int64_t hidden,
                            const int64_t *slice_width, int num_slices, int rank,
                            size_t workspace_bytes, int fp16, int paged);

/*
 * Copies the workspace's status word (LORA_STATUS_* bits OR-ed by every
 * lora_prepare_metadata since the last read) to *status, then clears it.
 * Synchronises `stream`.  Not capturable in a CUDA graph.
 */
int lora_read_status(void *workspace, uint32_t *status, void *stream);

/*
 * One layer - grouping, shrink and expand - without allocating anything.
 * The pages describe no counterpart to this call: it exists for callers that
 * cannot call cudaMalloc (a memory manager that owns the whole device, a
 * plugin host that hands out no device memory, code that must not allocate)
 * and so cannot provide the workspace the three calls above take.
 *
 * Arguments are those of lora_prepare_metadata, lora_shrink and lora_expand
 * (same meaning, layout and rules), minus the workspace; the caller still
 * passes every input and output, u and the three metadata arrays included.
 * `status` (optional, device pointer) receives this call's LORA_STATUS_* bits.
 *
 * The workspace is a file-scope device array of LORA_NOALLOC_SCRATCH_BYTES
 * (384 KB) in the library, which every GPU that loads the library holds
 * until the process exits.  It fits 8192 tokens with 128 adapters; sizes
 * whose workspace (lora_workspace_size) exceeds it are rejected with
 * LORA_ERR_WORKSPACE before anything is enqueued.  The first call on a
 * device looks up the array's device address (once per device, with that
 * device current): make that first call before any stream capture.  Every
 * call uses the same array and leaves its contents behind; the call clears
 * the status word it needs zeroed itself.  Calls that overlap on the GPU
 * (other streams, other threads) race on the array: serialise them.  Every
 * argument is checked before anything is enqueued.
 */
#define LORA_NOALLOC_SCRATCH_BYTES (384 * 1024)
int lora_apply_noalloc(const int32_t *token_lora_mapping, const int32_t *num_tokens,
                       int64_t max_num_tokens, int64_t max_loras, const uint16_t *x,
                       int64_t x_row_stride, int64_t hidden, const uint16_t *const *lora_a,
                       const uint16_t *const *lora_b, const int64_t *slice_width,
                       int num_slices, int rank, float scale, const float *lora_scales,
                       float *u, uint16_t *y, int64_t y_row_stride, int32_t *sorted_token_ids,
                       int32_t *num_tokens_per_lora, int32_t *lora_token_start_loc,
                       uint32_t *status, void *stream);

/* ------------------------------------------------------------------------
 * The operators of a decoder layer around its LoRA products: the norm whose
 * output a layer's product and lora_shrink read, and, behind the qkv product
 * that lora_expand completes, the append of k and v to a paged cache of 4-bit
 * values and the attention over it.  They keep the conventions above (device
 * pointers, static buffers of max_num_tokens rows with n valid ones, n in
 * device memory, stream order, no allocation, codes for bad arguments); where
 * a call takes `status`, it is NULL or a device word into which the call ORs
 * LORA_STATUS_* bits for what only the data reveals (lora_read_status reads and
 * clears it; the word must be 16-byte aligned for that).  16-bit data is bf16, or fp16 in the *_f16 forms.
 */

#define LORA_NORM_MAX_HIDDEN 32768

/*
 * Residual addition and root-mean-square norm, with the result in 16 bits
 * and / or in 8 bits with scales:
 *   z[t][h]     = x[t][h] + residual[t][h]                      (fp32)
 *   residual_out[t][h] = 16-bit(z[t][h])
 *   n[t][h]     = z[t][h] / sqrt(mean_h(z[t][h]^2) + eps) * weight[h]  (fp32)
 *   y[t][h]     = 16-bit(n[t][h])
 *   y8_scale[t][g] = max(max_{h in group g} |n[t][h]| * (1 / 448), 2^-100)
 *   y8[t][h]    = e4m3(n[t][h] / y8_scale[t][h / group]), the quotient rounded once
 *                 to fp32, then to the nearest, ties to even, saturating at 448
 * for t < n; rows t >= n are neither read nor written.  A NaN among a row's
 * z makes the row's n, scales and codes NaN.
 *
 *   x             16-bit[max_num_tokens][x_row_stride]
 *   residual      NULL (z = x), or 16-bit[max_num_tokens][residual_row_stride]
 *   residual_out  NULL, or where z goes; may be residual or x itself
 *   weight        16-bit[hidden]
 *   y             NULL, or 16-bit[max_num_tokens][y_row_stride] (y may be x)
 *   y8            NULL, or e4m3[max_num_tokens][y8_row_stride]
 *   y8_scale      fp32[max_num_tokens][hidden / group], given with y8
 *   group         columns per scale: hidden (one scale a row) or 128
 *   num_tokens    device int32: n (clamped to [0, max_num_tokens], which sets
 *                 LORA_STATUS_BAD_NUM_TOKENS)
 * Sizes: hidden a multiple of 8 up to LORA_NORM_MAX_HIDDEN (a multiple of 128
 * with groups of 128); 16-byte aligned pointers and row strides that are
 * multiples of 8 (y8: 8-byte aligned).  At least one of y, y8 and
 * residual_out is given.
 */
int lora_add_rmsnorm(const uint16_t *x, int64_t x_row_stride, const uint16_t *residual,
                     int64_t residual_row_stride, const uint16_t *weight, float eps,
                     int64_t hidden, uint16_t *residual_out, int64_t residual_out_row_stride,
                     uint16_t *y, int64_t y_row_stride, uint8_t *y8, int64_t y8_row_stride,
                     float *y8_scale, int64_t group, const int32_t *num_tokens,
                     int64_t max_num_tokens, uint32_t *status, void *stream);
int lora_add_rmsnorm_f16(const uint16_t *x, int64_t x_row_stride, const uint16_t *residual,
                         int64_t residual_row_stride, const uint16_t *weight, float eps,
                         int64_t hidden, uint16_t *residual_out,
                         int64_t residual_out_row_stride, uint16_t *y, int64_t y_row_stride,
                         uint8_t *y8, int64_t y8_row_stride, float *y8_scale, int64_t group,
                         const int32_t *num_tokens, int64_t max_num_tokens, uint32_t *status,
                         void *stream);

/*
 * The 4-bit paged cache.  One uint8 array, 16-byte aligned,
 *   cache[num_pages][num_kv_heads][page_size / 16][18 * head_dim]
 * where the last index is a block of 16 consecutive tokens of a page:
 *   [0, 8 D)      K codes, token r at r * D / 2: two e2m1 codes a byte, the even
 *                 dimension in the low nibble
 *   [8 D, 16 D)   V codes, the same
 *   [16 D, 17 D)  K scales, token r at r * D / 16: one e4m3 value for each 16
 *                 consecutive dimensions
 *   [17 D, 18 D)  V scales, the same
 * (D = head_dim, 64 or 128; 4.5 bits a value).  A value is e2m1(code) *
 * e4m3(scale) * k_scale or v_scale, a factor of the whole cache that the
 * calls take: choose it so that typical magnitudes land around 6 * 2^0 (the
 * scales cover 2^-9 .. 448).  Slot s of the cache is token s % page_size of page
 * s / page_size.  page_size is a multiple of 16 up to LORA_KV4_MAX_PAGE_SIZE.
 */
#define LORA_KV4_MAX_PAGE_SIZE 1024
#define LORA_KV4_MAX_SEQS 65536
#define LORA_KV4_MAX_HEADS 256

/*
 * Rotation of q and k by position, and the append of k and v to the cache:
 * for t < n with 0 <= position < max_positions
 *   q_out[t] = 16-bit(rot(q[t])),  cache slot slots[t] <- 4-bit(rot(k[t])), 4-bit(v[t])
 * rot turns the pair (a, b) of dimensions (i, i + rope_dim / 2), or (2 i, 2 i +
 * 1) when interleaved, into (a c - b s, b c + a s) with c = rope[pos][i] and
 * s = rope[pos][rope_dim / 2 + i], i < rope_dim / 2, in fp32 with each product
 * and sum rounded once; dimensions from rope_dim on stay.  4-bit() takes
 * 16 consecutive dimensions: with w = value * (1 / k_scale) (or v_scale),
 *   scale = e4m3(min(max|w| / 6, 448)),   code = e2m1(w / scale)
 * each to the nearest with ties to even, codes saturating at 6; where the
 * scale is 0 or NaN the codes are 0.  (A NaN among the 16 makes the scale NaN,
 * so all 16 read as NaN; an infinity reads as the largest value.)
 *
 *   q, q_out      NULL, or 16-bit[max_num_tokens][row stride], num_q_heads *
 *                 head_dim columns used; q_out may be q
 *   k, v          16-bit[max_num_tokens][row stride], num_kv_heads * head_dim
 *   rope          NULL (no rotation), or fp32[max_positions][rope_dim]
 *   positions     int32[max_num_tokens], given with rope
 *   slots         int32[max_num_tokens]; -1: the token's k and v are not
 *                 stored (its q is rotated all the same).  The slots of one
 *                 call must differ.
 *   k_held, v_held  NULL, or 16-bit[max_num_tokens][num_kv_heads * head_dim]
 *                 out: the values that the cache now stands for, written for
 *                 the stored tokens (for a caller that attends to the chunk it
 *                 has just appended without reading it back)
 * A position outside [0, max_positions) sets LORA_STATUS_BAD_POSITION and the
 * token is skipped altogether; a slot that is neither -1 nor inside the cache
 * sets LORA_STATUS_BAD_SLOT and the token's k and v are not stored.
 * Rows t >= n write nothing; what they hold may be read and is not used.
 * Sizes: rope_dim a multiple of 32 up to head_dim; strides multiples of 8;
 * pointers 16-byte aligned; num_pages * page_size below 2^31; the scales finite
 * and above 0.
 */
int lora_kv4_append(const uint16_t *q, int64_t q_row_stride, uint16_t *q_out,
                    int64_t q_out_row_stride, int num_q_heads, const uint16_t *k,
                    int64_t k_row_stride, const uint16_t *v, int64_t v_row_stride,
                    const float *rope, int64_t max_positions, int rope_dim, int interleaved,
                    const int32_t *positions, const int32_t *slots, uint8_t *cache,
                    int64_t num_pages, int num_kv_heads, int page_size, int head_dim,
                    float k_scale, float v_scale, uint16_t *k_held, uint16_t *v_held,
                    const int32_t *num_tokens, int64_t max_num_tokens, uint32_t *status,
                    void *stream);
int lora_kv4_append_f16(const uint16_t *q, int64_t q_row_stride, uint16_t *q_out,
                        int64_t q_out_row_stride, int num_q_heads, const uint16_t *k,
                        int64_t k_row_stride, const uint16_t *v, int64_t v_row_stride,
                        const float *rope, int64_t max_positions, int rope_dim, int interleaved,
                        const int32_t *positions, const int32_t *slots, uint8_t *cache,
                        int64_t num_pages, int num_kv_heads, int page_size, int head_dim,
                        float k_scale, float v_scale, uint16_t *k_held, uint16_t *v_held,
                        const int32_t *num_tokens, int64_t max_num_tokens, uint32_t *status,
                        void *stream);

/*
 * Causal attention of ragged rows of queries over the cache.  Sequence b has
 * the rows q_start[b] <= t < q_start[b + 1] of q and kv_len[b] keys (its rows'
 * own keys among them: they are appended first); its key j is slot
 * page_table[b][j / page_size] * page_size + j % page_size.  Row i of its m rows
 * stands at position p = kv_len[b] - m + i and sees the keys
 *   0 <= j <= p, and j > p - window where window > 0:
 *   x_j   = softmax_scale * q[t][h] . K[j][h / G]          G = num_q_heads / num_kv_heads
 *   out[t][h] = 16-bit( sum_j exp(x_j - m) V[j][h / G] / sum_j exp(x_j - m) )
 *   lse[t][h] = log sum_j exp(x_j)                         (fp32)
 * A row that sees no key gets 0 and lse = -inf.  One call serves single-token
 * decode, a few drafted tokens and chunks of prefill, mixed in one batch.
 *
 *   q, out        16-bit[max_num_tokens][row stride]; rows from
 *                 q_start[num_seqs] on are neither read nor written
 *   lse           NULL, or fp32[max_num_tokens][num_q_heads] out
 *   q_start       device int32[num_seqs + 1], ascending from 0
 *   kv_len        device int32[num_seqs]
 *   page_table    device int32[num_seqs][table_stride]; entries behind a
 *                 sequence's last page, and in front of the first page that
 *                 one of its rows' windows reaches, are not read
 *   max_q_len     a bound on the sequences' rows (host): it picks the kernels
 *   workspace     lora_kv4_attention_workspace_size bytes, 16-byte aligned,
 *                 zero-filled before its first use (every call leaves its
 *                 counters at zero); calls that share it run in one stream's order
 * Data that does not fit: a page id outside the cache masks its keys
 * (LORA_STATUS_BAD_SLOT); kv_len outside [0, table_stride * page_size] and rows
 * outside [0, max_num_tokens] are clamped and rows beyond max_q_len get no
 * output (LORA_STATUS_BAD_LENGTH).  What lies in the cache behind a sequence's
 * keys may hold anything, NaN scales included.
 * Sums, maxima and accumulators are fp32.  The products run on fp16 operands:
 * a cached value (without the cache's factor) is exact in fp16, a bf16 row of q
 * is scaled by a power of two so that its largest element lies in [2^14, 2^15)
 * (exact but for elements below 2^-29 of the row's largest), and a
 * probability is rounded once to fp16 (2^-11 of it; 2^-25 of the row's largest
 * where it lies below 2^-14 of that).  The weighted sum of V is accumulated in fp32
 * by the tensor cores, so a key may lose 2^-23 of the row's largest weight: a tail
 * of n keys of less weight than that each is counted in lse, and to within n 2^-23 in
 * out.  Scores may be of any size that fp32 holds.  A NaN among a row's keys,
 * or in its q, makes the row NaN; one in V the 16 dimensions of its scale; rows
 * that do not see that key keep their values.  Results do not depend on timing
 * or on what else is in the batch's workspace.  The kernels' waits are bounded
 * (200 ms): one that gives up sets LORA_STATUS_TIMEOUT, and the call's output is
 * unspecified; where `status` is NULL nothing else tells.
 */
size_t lora_kv4_attention_workspace_size(int64_t num_seqs, int64_t max_num_tokens,
                                         int64_t max_q_len, int num_q_heads, int num_kv_heads,
                                         int head_dim);
int lora_kv4_attention(const uint16_t *q, int64_t q_row_stride, uint16_t *out,
                       int64_t out_row_stride, float *lse, int num_q_heads, const uint8_t *cache,
                       int64_t num_pages, int num_kv_heads, int page_size, int head_dim,
                       float k_scale, float v_scale, const int32_t *q_start,
                       const int32_t *kv_len, const int32_t *page_table, int64_t table_stride,
                       int64_t num_seqs, int64_t max_num_tokens, int64_t max_q_len,
                       float softmax_scale, int64_t window, void *workspace,
                       size_t workspace_bytes, uint32_t *status, void *stream);
int lora_kv4_attention_f16(const uint16_t *q, int64_t q_row_stride, uint16_t *out,
                           int64_t out_row_stride, float *lse, int num_q_heads,
                           const uint8_t *cache, int64_t num_pages, int num_kv_heads,
                           int page_size, int head_dim, float k_scale, float v_scale,
                           const int32_t *q_start, const int32_t *kv_len,
                           const int32_t *page_table, int64_t table_stride, int64_t num_seqs,
                           int64_t max_num_tokens, int64_t max_q_len, float softmax_scale,
                           int64_t window, void *workspace, size_t workspace_bytes,
                           uint32_t *status, void *stream);

/* ------------------------------------------------------------------------
 * Drafted trees and bounded memory, over the same cache.  A step that verifies
 * drafted trees runs, behind the append of the drafted tokens: the attention of
 * the trees, lora_kv4_accept for the paths that the verification accepts,
 * and where the cache is bounded lora_kv4_key_weights and lora_kv4_evict.
 */

/*
 * lora_kv4_attention for the rows of drafted trees.  A sequence's m rows are the
 * drafted tokens, in any order, its last m keys theirs.  Row i sees
 *   the keys j < kv_len[b] - m in front of them (and j > p - window where window > 0,
 *     p = kv_len[b] - m + max(named - 1, 0) with the number of rows that its mask names), and
 *   key kv_len[b] - m + c where bit c of its mask is set: bit c % 32 of word c / 32, c < m.
 * A mask names a row's ancestors and the row itself, so that p is the row's position; nothing
 * else is assumed of it, and a row that sees no key gets 0 and lse = -inf.  The window hides keys
 * in front of the tree only: where it is shorter than the tree is deep, a row sees ancestors that
 * a row of lora_kv4_attention at its position would not.
 *
 *   tree_mask     device uint32[max_num_tokens][mask_words], 4-byte aligned; bits from m on
 *                 count for nothing
 *   mask_words    words of a row, 32 * mask_words >= max_q_len
 * All else, the workspace included, as in lora_kv4_attention.
 */
int lora_kv4_tree_attention(const uint16_t *q, int64_t q_row_stride, uint16_t *out,
                            int64_t out_row_stride, float *lse, int num_q_heads,
                            const uint8_t *cache, int64_t num_pages, int num_kv_heads,
                            int page_size, int head_dim, float k_scale, float v_scale,
                            const int32_t *q_start, const int32_t *kv_len,
                            const int32_t *page_table, int64_t table_stride, int64_t num_seqs,
                            int64_t max_num_tokens, int64_t max_q_len, const uint32_t *tree_mask,
                            int64_t mask_words, float softmax_scale, int64_t window,
                            void *workspace, size_t workspace_bytes, uint32_t *status,
                            void *stream);
int lora_kv4_tree_attention_f16(const uint16_t *q, int64_t q_row_stride, uint16_t *out,
                                int64_t out_row_stride, float *lse, int num_q_heads,
                                const uint8_t *cache, int64_t num_pages, int num_kv_heads,
                                int page_size, int head_dim, float k_scale, float v_scale,
                                const int32_t *q_start, const int32_t *kv_len,
                                const int32_t *page_table, int64_t table_stride,
                                int64_t num_seqs, int64_t max_num_tokens, int64_t max_q_len,
                                const uint32_t *tree_mask, int64_t mask_words,
                                float softmax_scale, int64_t window, void *workspace,
                                size_t workspace_bytes, uint32_t *status, void *stream);

#define LORA_KV4_MAX_PATH 512

/*
 * The accepted path of each sequence's tree: with n = kv_len[b] and m rows (q_start),
 *   key n - m + i  <-  key n - m + path[b][i]   for i < path_len[b], in every head,
 *   kv_len_out[b]   =  n - m + path_len[b].
 * Every key is read before any of its sequence is written, so a path may name rows in any
 * order and more than once.  Keys behind the path keep what they hold.
 *
 *   path          device int32[num_seqs][max_path], max_path up to LORA_KV4_MAX_PATH
 *   path_len      device int32[num_seqs]
 *   kv_len_out    device int32[num_seqs], apart from the other arrays
 * The pages of a sequence's last m keys hold no other sequence's.  Data that does not fit: lengths
 * are clamped (kv_len to the table, m to kv_len, path_len to m and max_path) and a path's row
 * outside [0, m) is not moved (LORA_STATUS_BAD_LENGTH); nothing is moved from or to a page
 * outside the cache (LORA_STATUS_BAD_SLOT).
 */
int lora_kv4_accept(uint8_t *cache, int64_t num_pages, int num_kv_heads, int page_size,
                    int head_dim, const int32_t *q_start, const int32_t *kv_len,
                    const int32_t *page_table, int64_t table_stride, int64_t num_seqs,
                    const int32_t *path, const int32_t *path_len, int64_t max_path,
                    int32_t *kv_len_out, uint32_t *status, void *stream);

#define LORA_KV4_MAX_KEYS ((1ll << 31) - 65536)

/*
 * The weight that each key has drawn: for every key head h and every key j of sequence b that
 * is one of its m rows' own (j >= kv_len[b] - m) or is seen by one of them,
 *   weights[b][h][j] = (j < kv_len[b] - m ? weights[b][h][j] : 0)
 *                      + sum over rows i that see j, heads g of h of exp(x_ijg - lse[t][g])
 * with x and the rows' sight as in lora_kv4_attention (causal, window), q and lse those of
 * that call.  The rows' own keys are new: their weight begins at 0, so weights needs no clearing.
 * With a path, the m rows are the tree's rows path[b][0 .. path_len[b]) in their order (q and lse
 * at q_start[b] + path[b][i]), and kv_len is that after lora_kv4_accept; they see what
 * lora_kv4_tree_attention has shown them: all rows of the path up to their own, and of the keys in front
 * what the window leaves.  Without one, they are all rows of the sequence.
 *
 *   weights       fp32[num_seqs][num_kv_heads][capacity], in and out
 *   lse           fp32[max_num_tokens][num_q_heads]; -inf: the row adds nothing, to a key of
 *                 NaN neither
 *   path, path_len  NULL, or int32[num_seqs][max_path] and int32[num_seqs]
 *   max_q_len     a bound on the rows that count (host): of the paths, where there are some; it picks
 *                 the kernels
 * Sums are fp32, for every key in an order that its sequence's rows and max_q_len settle, whatever
 * else is in the batch; products as in lora_kv4_attention.  A term exp(x - lse) is known to within 2^-16
 * of it times 1 + |lse| + softmax_scale * sum_d |q_d K_d| (an lse held in fp32 alone takes 2^-24 |lse|);
 * one below 2^-126 counts as 0; a sum of n terms and the weight before, none negative, loses n 2^-24 of it at
 * most.  A NaN in a row's q or lse makes the weights that it adds to NaN, one in a key that key's; q and
 * lse of rows of no sequence may hold anything.
 * Data that does not fit: as in lora_kv4_attention; keys from capacity
 * on have no weight, rows beyond max_q_len add nothing, nor does a path's row outside the
 * sequence's rows (LORA_STATUS_BAD_LENGTH).  A key whose page is outside the cache draws no
 * weight (LORA_STATUS_BAD_SLOT).
 */
int lora_kv4_key_weights(float *weights, int64_t capacity, const uint16_t *q,
                         int64_t q_row_stride, const float *lse, int num_q_heads,
                         const uint8_t *cache, int64_t num_pages, int num_kv_heads, int page_size,
                         int head_dim, float k_scale, const int32_t *q_start,
                         const int32_t *kv_len, const int32_t *page_table, int64_t table_stride,
                         int64_t num_seqs, int64_t max_num_tokens, int64_t max_q_len,
                         float softmax_scale, int64_t window, const int32_t *path,
                         const int32_t *path_len, int64_t max_path, uint32_t *status,
                         void *stream);
int lora_kv4_key_weights_f16(float *weights, int64_t capacity, const uint16_t *q,
                             int64_t q_row_stride, const float *lse, int num_q_heads,
                             const uint8_t *cache, int64_t num_pages, int num_kv_heads,
                             int page_size, int head_dim, float k_scale, const int32_t *q_start,
                             const int32_t *kv_len, const int32_t *page_table,
                             int64_t table_stride, int64_t num_seqs, int64_t max_num_tokens,
                             int64_t max_q_len, float softmax_scale, int64_t window,
                             const int32_t *path, const int32_t *path_len, int64_t max_path,
                             uint32_t *status, void *stream);

/*
 * Eviction by accumulated weight: a sequence of n = kv_len[b] > budget keys keeps budget of them in
 * each key head, each head its own.  key_pos[b][h][j] is the position of the token that key j
 * stands for, below 0 for a key that was appended since the last call; those become
 * last_pos[b] - (n - 1 - j).  The kept keys are first the protected ones, whose position is
 * below sink or above last_pos[b] - recent, then those of the largest weight (NaN below all
 * numbers); ties go to the lowest index.  The i-th kept key j >= budget, in the order of the indices,
 * takes the place of the i-th key j < budget that is not kept, with its weight and position;
 * the others stay where they are.  So keys of a head are in no order afterwards: attention
 * over them is called without a window.  key_pos of [budget, n) becomes -1.
 *   kv_len_out[b] = min(n, budget)
 * A sequence within its budget keeps everything; its new keys get their positions.
 *
 *   weights       fp32[num_seqs][num_kv_heads][capacity], in and out (lora_kv4_key_weights)
 *   key_pos       int32, the same; filled with -1 where a sequence begins
 *   last_pos      device int32[num_seqs]: the position of the last key's token
 *   budget        at least 1; sink + recent <= budget, both at least 0
 *   kv_len_out    device int32[num_seqs], apart from the other arrays
 * A sequence's pages hold no other sequence's.  Data that does not fit: kv_len is clamped to
 * the table and the capacity (LORA_STATUS_BAD_LENGTH); keys are not moved from or to a page
 * outside the cache (LORA_STATUS_BAD_SLOT), though their weights and positions are.
 */
int lora_kv4_evict(uint8_t *cache, int64_t num_pages, int num_kv_heads, int page_size,
                   int head_dim, float *weights, int32_t *key_pos, int64_t capacity,
                   const int32_t *kv_len, const int32_t *last_pos, const int32_t *page_table,
                   int64_t table_stride, int64_t num_seqs, int64_t budget, int64_t sink,
                   int64_t recent, int32_t *kv_len_out, uint32_t *status, void *stream);

/* Static text for a LORA_OK / LORA_ERR_* code. */
const char *lora_error_string(int code);

#ifdef __cplusplus
}
#endif

#endif /* GATHERED_RANK_GEMM_H */
