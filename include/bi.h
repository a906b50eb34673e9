/*
 * bi.h -- C ABI of libbi.so: batch-invariant reduction kernels for NVIDIA B200 (sm_100a).
 *
 * A kernel is batch-invariant when the bits it returns for one row of its input
 * do not depend on how many other rows share the call or where the row sits in
 * the batch.  The source pages state the property and its cause: inference
 * kernels such as matmul and RMSNorm reduce in an order shaped by the total
 * batch size, so a row's last bits change with the batch (readhandoff.com,
 * agent-run-reproducibility-pinning, "What does temperature zero actually
 * guarantee?"); the remedy is that the same input always takes the same
 * accumulation order (wiki.aimuse.me "Thinking Machines", batch-invariant
 * kernel section; glasp.co "How to achieve deterministic LLMs with batch
 * invariant inference", Key Insights), which rules out split-K and
 * shape-aware tiling (wiki.aimuse.me "Thinking Machines", section on the loss
 * of dynamic-batching optimisations).  The operations are those the public
 * library replaces -- mm, addmm, log_softmax, mean (ross.abutalabs.com
 * "thinking-machines-lab/batch_invariant_ops", "When to avoid") -- plus RMSNorm
 * and the SiLU-times-up glue of a gated MLP.
 *
 * How each entry point fixes its order (the same for every M):
 *   - bi_matmul / bi_addmm: tcgen05/TMEM tiles fed by TMA; the tile width is a
 *     function of the weight's shape alone (bi_gemm_config), never of M; every
 *     output element accumulates its K products in fp32, 16 at a time, in
 *     ascending K, in every configuration; no split-K, no stream-K.
 *   - bi_rmsnorm / bi_mean / bi_log_softmax: each row is reduced by one thread
 *     block (for long-row means, persistent blocks take rows in turn); the
 *     block size and each thread's element set depend only on the row length;
 *     partial results merge through a fixed warp-shuffle tree and a fixed
 *     cross-warp tree.
 *   - bi_paged_decode_attention / bi_token_logprobs: cuts fixed by the sequence's own length
 *     or the row's; how many blocks share the pieces may follow the batch, their order of folding
 *     does not.
 *
 * Conventions shared by every entry point
 *   - Tensors are row-major.  Pointers marked "device" point to global memory
 *     of the current CUDA device; the caller allocates, owns and frees every
 *     buffer.  The library allocates no device memory in any call.
 *   - `stream` is a cudaStream_t passed as `void *` (so that this header needs no CUDA
 *     header; NULL = the legacy default stream).  Calls are
 *     asynchronous on that stream.  Argument errors are returned before anything
 *     is launched; a launch failure returns BI_ERR_CUDA.  The status is the result of this
 *     call's own launches: an error left by another library's earlier launch on the thread
 *     is neither reported nor cleared (apart from a context-wide fault, which fails every
 *     launch).  The GEMM, RMSNorm, mean,
 *     one-block log_softmax, decode-attention (dense and paged), rotation, append and token
 *     log-probability kernels are launched with programmatic stream serialization:
 *     they may start their on-chip set-up while the previous kernel on the stream drains,
 *     and read or write global memory only after that kernel has completed, so stream
 *     order holds as for any launch.
 *   - M = 0 (no rows) is a no-op that returns BI_OK.
 *   - Outputs must not overlap inputs, except where an entry point allows an input as its output.
 *   - bf16 is IEEE-style bfloat16 (1-8-7); every bf16 output is rounded once,
 *     to nearest-even, from an fp32 value.
 *   - The library keeps per-device state for the life of the process (the SM count, the
 *     status word's address, kernel attributes, the no-allocation array's address) and a
 *     cache of encoded TMA tensor maps keyed by (base address, extents, row stride, box).
 *     Calls across a cudaDeviceReset of a device the library has already used are not
 *     supported: the cached device addresses belong to the context that reset destroyed.
 *   - Every device-side wait is bounded; a wait that runs out records
 *     BI_ERR_TIMEOUT in a per-device status word, the kernel releases what it
 *     holds and returns.  Read it with bi_get_device_status.
 */
#ifndef BI_H
#define BI_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    BI_OK = 0,
    BI_ERR_INVALID_ARG = 1,  /* null pointer, negative size, leading dim too small, bad enum */
    BI_ERR_UNSUPPORTED = 2,  /* a size the kernels do not handle (e.g. > 2^31-1 rows)        */
    BI_ERR_ALIGNMENT = 3,    /* base pointer or leading dimension breaks the 16-byte rule   */
    BI_ERR_CUDA = 4,         /* a CUDA runtime/driver call or a launch failed                */
    BI_ERR_TIMEOUT = 5       /* a bounded device-side wait ran out (reported via the status) */
} bi_status;

typedef enum { BI_BF16 = 0, BI_F32 = 1 } bi_dtype;

typedef enum {
    BI_B_KN = 0, /* B stored [K, N] row-major: the right operand of torch.mm           */
    BI_B_NK = 1  /* B stored [N, K] row-major: an nn.Linear weight (C = A . B^T)       */
} bi_b_layout;

/*
 * bi_matmul -- C = A . B  (torch.mm; for BI_B_NK, torch.nn.functional.linear without bias).
 * Passage: ross.abutalabs.com "thinking-machines-lab/batch_invariant_ops", "When to
 * avoid" (mm is covered) and "Use cases" (matrix multiplication gives the same output
 * for different batch sizes).
 *
 *   A  device, bf16, [M, K], leading dimension lda >= K (elements)
 *   B  device, bf16, [K, N] with ldb >= N (BI_B_KN) or [N, K] with ldb >= K (BI_B_NK)
 *   C  device, [M, N], leading dimension ldc >= N, element type c_dtype (BI_BF16 or BI_F32)
 *   C[i][j] = round_{c_dtype}( sum_{k ascending} A[i][k] * B(k, j) ), products and sums in fp32.
 *   K = 0 writes zeros.
 * Alignment: A, B, C base addresses 16-byte aligned; lda, ldb multiples of 8 elements;
 *   ldc a multiple of 8 (bf16) or 4 (f32) elements.  Otherwise BI_ERR_ALIGNMENT.
 * Limits: M, N, K <= 2^31 - 1; otherwise BI_ERR_UNSUPPORTED.
 */
bi_status bi_matmul(const void *A, int64_t lda, const void *B, int64_t ldb, bi_b_layout b_layout,
                    void *C, int64_t ldc, bi_dtype c_dtype, int64_t M, int64_t N, int64_t K,
                    void *stream);

/*
 * bi_addmm -- C = input + A . B  (torch.addmm with alpha = beta = 1).
 * Passage: ross.abutalabs.com "thinking-machines-lab/batch_invariant_ops", "When to
 * avoid" (addmm is covered).
 *
 *   input  device, bf16.  ld_input == 0: a bias vector [N] added to every row.
 *          ld_input >= N: a matrix [M, N] (e.g. a residual) with that leading dimension,
 *          which must be a multiple of 8; base 16-byte aligned.
 *   The input is widened to fp32 and added to the fp32 accumulator once, after the last
 *   product, before the single rounding to c_dtype.  All else as bi_matmul.
 */
bi_status bi_addmm(const void *input, int64_t ld_input, const void *A, int64_t lda, const void *B,
                   int64_t ldb, bi_b_layout b_layout, void *C, int64_t ldc, bi_dtype c_dtype,
                   int64_t M, int64_t N, int64_t K, void *stream);

/*
 * bi_matmul_silu_mul -- H = silu(A . Wg) * (A . Wu): the gate/up projection of a gated MLP
 * with the SiLU-times-up glue applied in the GEMM's epilogue, so the [M, 2F] gate/up
 * activations never reach memory.  Elementwise glue after the same batch-invariant
 * reduction as bi_matmul; not an operation the pages name (the MLP block of the workload).
 *
 *   A  device, bf16, [M, K], lda >= K.
 *   B  device, bf16, the gate and up weights stacked: BI_B_NK: [2F, K] with rows [0, F) the
 *      gate and rows [F, 2F) the up projection (ldb >= K); BI_B_KN: [K, 2F] with columns
 *      [0, F) gate and [F, 2F) up (ldb >= 2F).
 *   H  device, bf16, [M, F], ldh >= F.
 *   g and u are the fp32 accumulators of bi_matmul (same K order); h = (g / (1 + exp(-g))) * u
 *   in fp32, one rounding to bf16.  (bi_matmul followed by bi_silu_mul rounds g and u to bf16
 *   first, so the two paths agree to the bf16 tolerance, not bit for bit.)
 *   Alignment and limits as bi_matmul; 2F <= 2^31 - 1; with BI_B_KN, F must also be a multiple
 *   of 8 (the up half starts at column F), else BI_ERR_ALIGNMENT.  K = 0 writes zeros.
 */
bi_status bi_matmul_silu_mul(const void *A, int64_t lda, const void *B, int64_t ldb,
                             bi_b_layout b_layout, void *H, int64_t ldh, int64_t M, int64_t F,
                             int64_t K, void *stream);

/*
 * bi_rmsnorm -- y = x * r * w,  r = 1 / sqrt( sum_j x_j^2 / H + eps ), per row.
 * Passage: readhandoff.com agent-run-reproducibility-pinning, "What does temperature
 * zero actually guarantee?" and the FAQ (RMSNorm is one of the kernels whose result
 * depends on the batch by default).
 *
 *   x  device, bf16, [M, H] contiguous;  w device, bf16, [H];  y device, bf16, [M, H].
 *   fp32 arithmetic inside; one rounding of (x * r) * w to bf16.  eps >= 0.
 *   x, w, y 16-byte aligned when H is a multiple of 8 (the vector path), else any alignment.
 */
bi_status bi_rmsnorm(const void *x, const void *w, void *y, int64_t M, int64_t H, float eps,
                     void *stream);

/*
 * bi_mean -- y_i = ( sum_j x_ij ) / H, per row (torch.mean over the last dimension).
 * Passage: ross.abutalabs.com "thinking-machines-lab/batch_invariant_ops", "When to
 * avoid" (mean is covered); trustbutveri.fyi "Evidence & limits", Evidence (SGLang
 * integrated the mean kernel).
 *
 *   x  device, fp32, [M, H] contiguous;  y device, fp32, [M].
 *   fp32 sum in a fixed tree, then one IEEE division by H.
 *   x 16-byte aligned when H is a multiple of 4 (the vector path).
 */
bi_status bi_mean(const float *x, float *y, int64_t M, int64_t H, void *stream);

/*
 * bi_log_softmax -- y_j = (x_j - m) - log( sum_k exp(x_k - m) ),  m = max_k x_k, per row.
 * Passage: ross.abutalabs.com "thinking-machines-lab/batch_invariant_ops", "When to
 * avoid" (log_softmax is covered); trustbutveri.fyi "Evidence & limits", Evidence.
 *
 *   x  device, [M, V] contiguous, x_dtype BI_F32 or BI_BF16 (bf16 is widened exactly);
 *   y  device, fp32, [M, V].
 *   One thread block per row.  Per-thread running (max, sum) pairs merged through a fixed
 *   tree; the row is read twice (once for the statistics, once to write y; the last chunks of
 *   the first pass are still in shared memory for the second).
 *   x and y 16-byte aligned when V is a multiple of 8 (bf16) / 4 (f32), the vector path.
 */
bi_status bi_log_softmax(const void *x, bi_dtype x_dtype, float *y, int64_t M, int64_t V,
                         void *stream);

/*
 * bi_log_softmax_cluster -- the same y as bi_log_softmax, for long rows, computed by a cluster of
 * 4 CTAs per row (an opt-in variant: bi_log_softmax keeps one CTA per row).  Passage: as
 * bi_log_softmax.  The row is cut into 4 slices of S = 8 * ceil(V / 32) elements, a cut fixed by V
 * alone; each CTA bulk-copies its slice into shared memory, reduces it to a (max, sum of exp)
 * pair, and every CTA folds the 4 pairs in rank order (distributed shared memory) before
 * writing its slice of y from shared memory, so the row is read from memory once.  The result
 * is batch-invariant; it is a different fixed order from bi_log_softmax's, so the two agree to
 * the tolerance, not bit for bit.
 *
 *   x, x_dtype, y, M, V as bi_log_softmax; x and y 16-byte aligned.
 *   Rows it takes: V % 8 == 0 (bf16) or V % 4 == 0 (fp32), V * element size >= 64 KiB and
 *   S * element size <= 96 KiB, i.e. 32768 <= V <= 196608 for bf16 and 16384 <= V <= 98304 for
 *   fp32.  Any other V returns BI_ERR_UNSUPPORTED without launching.
 */
bi_status bi_log_softmax_cluster(const void *x, bi_dtype x_dtype, float *y, int64_t M, int64_t V,
                                 void *stream);

/*
 * bi_log_softmax_split -- the same y as bi_log_softmax, computed by many blocks per row, for
 * short batches (decode-time sampling) where one block per row leaves most SMs idle.
 * Passage: as bi_log_softmax.  The row is cut into chunks of 4096 elements, a cut fixed by V
 * alone; each chunk is reduced to a (max, sum of exp) partial, and every block of the row
 * merges the row's partials in one fixed tree before writing its chunk.  The result is
 * batch-invariant; it is a different fixed order from bi_log_softmax's, so the two agree to
 * the tolerance, not bit for bit.
 *
 *   x, x_dtype, y, M, V as bi_log_softmax; V must be a multiple of 8 (else
 *   BI_ERR_UNSUPPORTED), x and y 16-byte aligned; M <= 65535.
 *   scratch  device memory owned by the caller, 16-byte aligned, at least
 *            bi_log_softmax_split_scratch_bytes(M, V) bytes; overwritten by the call (two
 *            launches on `stream`), so calls that overlap on the GPU need separate scratch.
 *   Too small a scratch returns BI_ERR_INVALID_ARG.
 */
bi_status bi_log_softmax_split(const void *x, bi_dtype x_dtype, float *y, int64_t M, int64_t V,
                               void *scratch, size_t scratch_bytes, void *stream);

/* Bytes of scratch bi_log_softmax_split needs for M rows of V elements (0 if M or V <= 0). */
size_t bi_log_softmax_split_scratch_bytes(int64_t M, int64_t V);

/*
 * bi_log_softmax_split_noalloc -- bi_log_softmax_split for callers that cannot allocate
 * device memory at call time: ones working inside a device-memory budget reserved up front
 * by a pool they do not own, plugins whose host framework controls every allocation, or hot
 * paths that cannot afford the synchronisation a cudaMalloc implies.  The paper has no
 * counterpart; this is a library convenience.
 *
 * The per-(row, chunk) partials live in a fixed array inside libbi.so's device image (512 KiB,
 * 65536 partials) instead of caller scratch.  Every GPU that loads the library holds that
 * array until the process exits; no call allocates or frees anything.
 *
 *   x, x_dtype, y, M, V as bi_log_softmax_split (V a multiple of 8, 16-byte aligned x and y,
 *   M <= 65535).  Limit: M * ceil(V / 4096) <= 65536 (e.g. M <= 1724 rows at V = 151936);
 *   larger calls return BI_ERR_UNSUPPORTED without launching.
 *   The result is the same as bi_log_softmax_split's for the same input.
 *   The first call on a device looks up the array's device address (once per device, with
 *   that device current); make that first call before capturing any stream.
 *   All calls on a device share the one array, and it keeps the last call's partials (every
 *   call overwrites all the partials it reads, so nothing has to start at zero).  Calls that
 *   overlap on the GPU -- on different streams without ordering between them -- race on it.
 */
bi_status bi_log_softmax_split_noalloc(const void *x, bi_dtype x_dtype, float *y, int64_t M,
                                       int64_t V, void *stream);

/*
 * bi_silu_mul -- h_ij = silu(g_ij) * u_ij with g = gu[:, 0:F], u = gu[:, F:2F],
 * silu(g) = g / (1 + exp(-g)).  Elementwise glue of a gated MLP (no reduction, so
 * batch-invariant by construction); not an operation the pages name.
 *
 *   gu device, bf16, [M, 2F] contiguous;  h device, bf16, [M, F].
 *   fp32 inside, one rounding to bf16.  16-byte aligned when F is a multiple of 8.
 */
bi_status bi_silu_mul(const void *gu, void *h, int64_t M, int64_t F, void *stream);

/*
 * bi_decode_attention -- one decode step of softmax attention with grouped-query heads:
 * for each sequence b and query head h (reading kv head h / (Hq / Hkv)),
 *   s_t = scale * q[b,h,:] . k[b,t,g,:],  p = softmax over t < seq_lens[b],  out[b,h,:] = sum_t p_t v[b,t,g,:].
 * Passage: trustbutveri.fyi "Evidence & limits", Evidence and Limitations (SGLang wrote
 * batch-invariant attention kernels; an improved attention kernel took the deterministic
 * Qwen3-8B run from 55 s to 42 s); readhandoff.com agent-run-reproducibility-pinning,
 * "What does temperature zero actually guarantee?" (attention is not batch-invariant by
 * default).
 *
 * Batch invariance: each sequence's cache is cut into splits of 512 tokens, a cut fixed by
 * its own length (never by the batch size or the GPU's occupancy, unlike split-KV decoding
 * that sizes splits to fill the machine).  Per split, scores are fp32 dot products over D in
 * ascending order; the split is taken in four 128-token pieces in ascending order, each
 * raising a running maximum by a fixed tree and rescaling the sums of exp(s - max) and the
 * weighted value sums accumulated so far, which run over tokens in ascending order; the
 * splits are then folded in ascending order.  A sequence's output does not depend on the
 * other sequences in the batch.
 *
 *   q        device, bf16, [B, Hq, D];  out device, bf16, [B, Hq, D] (one rounding).
 *   k_cache, v_cache  device, bf16, [B, Lmax, Hkv, D]; only the first seq_lens[b] tokens of
 *            sequence b are read.
 *   seq_lens device, int32, [B], each in 1 .. Lmax.  A value outside is clamped and
 *            BI_ERR_INVALID_ARG is recorded in the device status word.
 *   D must be 64 or 128 and Hq / Hkv one of 1, 2, 4, 8 (else BI_ERR_UNSUPPORTED); B, Hq, Hkv <= 65535
 *   and B * Hkv * ceil(Lmax / 512) < 2^31 (else BI_ERR_UNSUPPORTED).
 *   scratch  caller-owned device memory, 16-byte aligned, at least
 *            bi_decode_attention_scratch_bytes(B, Hq, D, Lmax) bytes; overwritten (two
 *            launches on `stream`; one when Lmax <= 512, where every sequence is one split
 *            and the first launch writes out itself), so overlapping calls need separate
 *            scratch.
 *   q, caches 16-byte aligned; seq_lens 4-byte aligned.
 */
bi_status bi_decode_attention(const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *seq_lens, void *out, int64_t B, int64_t Hq, int64_t Hkv,
                              int64_t D, int64_t Lmax, float scale, void *scratch, size_t scratch_bytes,
                              void *stream);

/* Bytes of scratch bi_decode_attention needs (0 if any size is <= 0). */
size_t bi_decode_attention_scratch_bytes(int64_t B, int64_t Hq, int64_t D, int64_t Lmax);

/*
 * bi_rope -- rotary positions: y = x with the first R entries of every head turned by its token's
 * position.  Pair number i < R/2 of head h of token t, entries (a, b) of x, becomes
 *   (a cos w - b sin w, b cos w + a sin w) * scale,   w = positions[t] * inv_freq[i],
 * and entries R .. D-1 are copied as they are.  `inverse` turns by -w: the transposed map, which is
 * the gradient of the forward one.  Elementwise, so batch-invariant by construction; not an
 * operation the pages name (the attention input of the workload's model).
 *
 *   x, y       device, [T, H, D] of x_dtype (bf16 or fp32), entries of a head consecutive, tokens and
 *              heads token_stride / head_stride elements apart (any strides >= 0 for x; those of y
 *              must keep its heads apart).  y may be x itself with the same strides.
 *   positions  device, int32, [T], any sign.
 *   inv_freq   device, fp64, [R/2] (bi_rope_freqs).  R even, 0 <= R <= D <= 1024.  R = 0: nothing is turned, and positions
 *              and inv_freq may be NULL.
 *   layout     BI_ROPE_HALF: pair i is entries (i, i + R/2); BI_ROPE_INTERLEAVED: (2i, 2i + 1).
 *   The angle is an fp64 product reduced to a fraction of a turn, so far positions keep their
 *   digits; cosines and sines are within 1.5 * 2^-24 and the rest is fp32 with one rounding to bf16.  Heads move in
 *   16-byte pieces where R/2, the strides and the addresses are multiples of them.  Where R/2 is not but D is, they move so
 *   too and the pairs are turned in shared memory, but for some calls in place, where the turned entries alone move.  Else
 *   pairs move two entries or one at a time, and entries R .. D-1 in the widest pieces that fit them.  The bits are the
 *   same.
 *   T <= 2^31 - 1, H <= 65535.
 */
typedef enum { BI_ROPE_HALF = 0, BI_ROPE_INTERLEAVED = 1 } bi_rope_layout;

bi_status bi_rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, void *y, int64_t y_token_stride,
                  int64_t y_head_stride, bi_dtype x_dtype, const int32_t *positions, const double *inv_freq,
                  int64_t T, int64_t H, int64_t D, int64_t R, bi_rope_layout layout, float scale, int inverse,
                  void *stream);

/*
 * bi_rope_freqs -- the inverse frequencies theta^(-2i/R), i < R/2, and the output scale of a scaled
 * variant, in host memory (no device is touched).  kind and params:
 *   BI_ROPE_PLAIN   none.  scale 1.
 *   BI_ROPE_LINEAR  {factor}: every frequency / factor.  scale 1.
 *   BI_ROPE_NTK     {factor}: theta replaced by theta * factor^(R / (R - 2)) (R > 2).  scale 1.
 *   BI_ROPE_YARN    {factor, original length, beta_fast, beta_slow}: frequency i is blended from f (more than
 *                   beta_fast turns within the original length) to f / factor (fewer than beta_slow) by a
 *                   linear ramp over i between the two bounds, floor and ceiling of
 *                   R log(length / (2 pi beta)) / (2 log theta), the lower at least 0, the upper at most R - 1; with all
 *                   pairs on one side of both, all are kept or all divided.  scale 0.1 log(factor) + 1.
 *   BI_ROPE_BANDED  {factor, original length, low, high}: wavelengths shorter than length / high keep f, longer than
 *                   length / low get f / factor, between them the two are blended linearly in
 *                   length / wavelength.  scale 1.
 * theta > 1, factor >= 1, lengths > 0, beta_fast > beta_slow > 0, high > low > 0; otherwise BI_ERR_INVALID_ARG.
 */
typedef enum {
    BI_ROPE_PLAIN = 0,
    BI_ROPE_LINEAR = 1,
    BI_ROPE_NTK = 2,
    BI_ROPE_YARN = 3,
    BI_ROPE_BANDED = 4
} bi_rope_kind;

bi_status bi_rope_freqs(int64_t R, double theta, bi_rope_kind kind, const double *params, int64_t n_params,
                        double *inv_freq, double *scale);

/*
 * A paged key/value cache: `pages` pages of page_size tokens, bf16.  Entry d of head h of row r of page
 * g is k[g * page_stride + r * token_stride + h * head_stride + d] (strides in elements, the same for
 * v), so [pages, page_size, heads, D], [pages, heads, page_size, D] and keys beside values in one
 * buffer are all described.  A sequence's tokens p = 0, 1, ... sit in row p % page_size of page
 * block_table[b][p / page_size].  k and v 16-byte aligned, strides multiples of 8.
 */
typedef struct {
    void *k, *v;
    int64_t pages, page_size, heads, head_dim;
    int64_t page_stride, token_stride, head_stride;
} bi_paged_cache;

/*
 * bi_paged_append -- write new tokens' keys and values into a paged cache, the keys turned as bi_rope
 * turns them, and optionally turn the same tokens' queries.  Elementwise, batch-invariant by
 * construction; not an operation the pages name (the step before bi_paged_decode_attention).
 *
 *   k, v        device, bf16, [T, heads, D], token and head strides as in bi_rope.
 *   q, q_out    device, bf16, [T, Hq, D], or both NULL; q_out may be q with the same strides.
 *   cu_new      device, int32, [B+1], ascending: the new tokens of sequence b are cu_new[b] .. cu_new[b+1]-1.
 *               NULL: T = B, one each.
 *   seq_lens    device, int32, [B]: tokens of each sequence with the new ones, which come last: token t
 *               of sequence b takes place seq_lens[b] - (cu_new[b+1] - t).
 *   block_table device, int32, [B, max_pages], rows table_stride elements apart.
 *   positions   device, int32, [T]: what turns each token, or NULL: its place.
 *   inv_freq    device, fp64, [R/2], as in bi_rope; R = 0: nothing is turned (NULL).
 * Tokens behind cu_new[B] (or before cu_new[0]) and those of a sequence with seq_lens[b] = 0 are skipped:
 * nothing of theirs is read back or written.  A place that is negative or past the table, or a page
 * outside 0 .. pages-1, records BI_ERR_INVALID_ARG in the device status word and skips the token.
 * Two tokens must not share a place: pages that receive tokens belong to one sequence.  (Where two do, each
 * entry there is one of theirs, which one is not defined.)
 * D <= 1024, heads and Hq <= 65535, T, B < 2^31, pages and page_size <= 2^31 - 1.
 * Pieces as in bi_rope between two tensors; k, v, q need no alignment beyond their type's.
 */
bi_status bi_paged_append(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                          int64_t v_token_stride, int64_t v_head_stride, const void *q, int64_t q_token_stride,
                          int64_t q_head_stride, void *q_out, int64_t q_out_token_stride,
                          int64_t q_out_head_stride, int64_t Hq, const bi_paged_cache *cache,
                          const int32_t *block_table, int64_t table_stride, int64_t max_pages,
                          const int32_t *seq_lens, const int32_t *cu_new, const int32_t *positions,
                          const double *inv_freq, int64_t R, bi_rope_layout layout, float scale, int64_t T,
                          int64_t B, void *stream);

/*
 * bi_paged_decode_attention -- bi_decode_attention over a paged cache: for each sequence b and query head
 * h (reading kv head h / (Hq / heads)), out[b,h,:] = sum_t p_t v_t with p = softmax(scale * q[b,h,:] . k_t)
 * over the sequence's t < seq_lens[b].  A sequence of length 0 (an empty place of a padded batch) gets zeros.
 * Passage: as bi_decode_attention.
 *
 * Batch invariance: a sequence is one split up to 512 tokens and splits of 256 beyond, in tiles of 32, cuts
 * fixed by its own length; scores are fp32 dot products, four chains take a split's tiles w, w + 4, ... under
 * a running maximum and are folded in order, and splits in a tree fixed by their number.  The weights keep their fp32 bits.  A
 * sequence's output does not depend on the others, on where its pages lie, on the page size or on max_len.  Keys and values
 * of its own tokens should be finite (an infinite value gives NaN); what lies past its end may be anything.
 *
 *   q        device, bf16, [B, Hq, D], heads consecutive, sequences q_stride elements apart (a multiple of 8).
 *   out      device, bf16, [B, Hq, D] contiguous (one rounding).
 *   seq_lens device, int32, [B], each in 0 .. max_len.  A value outside is clamped and BI_ERR_INVALID_ARG
 *            recorded in the device status word.
 *   block_table as in bi_paged_append; only the entries of a sequence's own tokens are read.  A page outside
 *            0 .. pages-1 records BI_ERR_INVALID_ARG and its tokens count with keys and values of zero.
 *   max_len  what the host knows of the longest sequence, 1 .. max_pages * page_size.
 *   D must be 64 or 128 and Hq / heads 1 .. 16, any page_size >= 1 (else BI_ERR_UNSUPPORTED; pages of fewer
 *   than 8 tokens, or of an odd number, take more and smaller copies); B, Hq <= 65535 and
 *   min(B, 2048) * heads * ceil(max_len / 256) < 2^31.
 *   scratch  caller-owned device memory, 16-byte aligned, bi_paged_decode_attention_scratch_bytes bytes;
 *            overwritten (two launches on `stream` per 2048 sequences; one when max_len <= 512), so
 *            overlapping calls need separate scratch.
 *   q, out 16-byte aligned.
 */
bi_status bi_paged_decode_attention(const void *q, int64_t q_stride, const bi_paged_cache *cache,
                                    const int32_t *block_table, int64_t table_stride, int64_t max_pages,
                                    const int32_t *seq_lens, void *out, int64_t B, int64_t Hq, int64_t max_len,
                                    float scale, void *scratch, size_t scratch_bytes, void *stream);

/* Bytes of scratch bi_paged_decode_attention needs (0 if any size is <= 0 or max_len <= 512). */
size_t bi_paged_decode_attention_scratch_bytes(int64_t B, int64_t Hq, int64_t D, int64_t max_len);

/*
 * bi_token_logprobs -- what sampling and scoring keep of bi_log_softmax, without writing [M, V] values.
 * Per row, with z = scale * x (scale = 1 / temperature) and y = z - logsumexp(z):
 *   logprobs_i = y[tokens_i],  entropy_i = -sum_j exp(y_j) y_j (0 where exp(y_j) = 0),
 *   logsumexp_i, and the top_k largest y_j with their tokens, in descending order, equal logits in
 *   ascending token order.
 * Passage: as bi_log_softmax.
 *
 *   x        device, [M, V] of x_dtype (bf16 or fp32), rows ldx >= V elements apart.
 *   tokens   device, int32, [M].  A negative one is not scored (logprob 0); one >= V gives NaN and records
 *            BI_ERR_INVALID_ARG in the device status word.
 *   logprobs, entropy, logsumexp  device, fp32, [M]; each may be NULL (tokens may be when logprobs is).
 *   top_logprobs, top_tokens  device, fp32 / int32, [M, top_k]; 0 <= top_k <= min(32, V).
 *   -inf logits are masked entries.  A row of only -inf has logsumexp -inf and NaN elsewhere; +inf or NaN
 *   in a row makes its values NaN.  NaN logits rank below all others.
 *   1 <= V <= 262144.  scale > 0, finite.  Rows of any alignment; 16-byte aligned rows are read faster.
 * Batch invariance: a row is cut into pieces of 8192 (bf16) or 4096 (fp32) elements, each reduced in one
 * fixed order by one block and folded in one fixed tree.  How many blocks share a row's pieces depends on
 * M and changes no bit.
 */
bi_status bi_token_logprobs(const void *x, int64_t ldx, bi_dtype x_dtype, const int32_t *tokens, float scale,
                            int64_t top_k, float *logprobs, float *entropy, float *logsumexp, float *top_logprobs,
                            int32_t *top_tokens, int64_t M, int64_t V, void *stream);

/*
 * bi_get_device_status -- synchronise `stream`, then read and clear the current
 * device's status word.  *out receives BI_OK or the first error a kernel recorded
 * since the last read (BI_ERR_TIMEOUT for a bounded wait that ran out, BI_ERR_INVALID_ARG for a length, page,
 * place or token that a kernel found out of range).
 * Returns BI_ERR_CUDA if the synchronisation or the read fails.
 */
bi_status bi_get_device_status(void *stream, int32_t *out);

/*
 * bi_selftest_wait_timeout -- launch one block that waits on a shared-memory
 * barrier nothing will complete, through the same bounded wait the GEMM uses,
 * with the given limit (nanoseconds, 1000 .. 10^10).  The wait gives up, records
 * BI_ERR_TIMEOUT in the status word and the kernel returns normally; the device
 * context stays usable.  For testing the failure path without a GPU fault.
 */
bi_status bi_selftest_wait_timeout(int64_t limit_ns, void *stream);

/* Human-readable name of a status code (static storage; never NULL). */
const char *bi_status_string(bi_status status);

/*
 * bi_gemm_config -- report the tile configuration the GEMM entry points use for a
 * weight of `weight_rows` rows in [N, K] (BI_B_NK) storage: N for bi_matmul /
 * bi_addmm, 2F for bi_matmul_silu_mul.  It reports the output tile bm x bn, K per
 * pipeline stage bk, the number of stages, and the K step of one tensor-core
 * instruction.  bn is 128 up to 1024 rows. Above that it is 192 where 192-column
 * tiles fill the B200's CTA pairs in fewer cost-weighted waves than 256-column tiles
 * for a 1024-row batch (e.g. 6144 or 24576 rows), else 256. [K, N] (BI_B_KN)
 * weights run bn = 256 where this reports 192.  The configuration depends on the
 * weight alone -- every M of a given weight runs the same one -- and all
 * configurations take the same 16-wide K steps in ascending order, so an element's
 * bits do not depend on it.  weight_rows <= 0 reports bn = 256.  Any pointer may be NULL.
 */
void bi_gemm_config(int64_t weight_rows, int32_t *bm, int32_t *bn, int32_t *bk, int32_t *stages, int32_t *mma_k);

/*
 * bi_tensor_map_cache_stats -- how many TMA tensor-map look-ups of the GEMM entry points were
 * served from the library's cache (*hits) and how many had to be encoded (*misses) since the
 * library was loaded.  A GEMM call looks up two maps (weights and activations), keyed by
 * (base address, extents, row stride, box); a repeated call with the same buffers hits twice.
 * Either pointer may be NULL.
 */
void bi_tensor_map_cache_stats(int64_t *hits, int64_t *misses);

/* Library version as major*10000 + minor*100 + patch. */
int32_t bi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* BI_H */
