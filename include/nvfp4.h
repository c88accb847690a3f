/*
 * nvfp4.h -- C ABI of the GB300 (sm_103a) NVFP4 / MXFP4 block-scaled GEMM library.
 *
 * Operations (each entry point cites the passage that defines it):
 *   nvfp4_quantize      bf16 -> NVFP4 (packed e2m1 + e4m3 scale per 16, 128x4 swizzled scales)
 *   nvfp4_gemm          D[M,N] = alpha * deq(A) deq(B)^T, bf16 out, fp32 accumulation
 *                       (+ nvfp4_gemm_plan, nvfp4_gemm_workspace_size, nvfp4_gemm_noalloc)
 *   nvfp4_quantize_gemm nvfp4_quantize of the activation fused into nvfp4_gemm (M <= 256)
 *   mxfp4_quantize      bf16 -> MXFP4 (packed e2m1 + ue8m0 scale per 32), optionally grouped by expert
 *   mxfp4_grouped_gemm  per-expert D_e = alpha * deq(A_e) deq(B_e)^T for MoE experts
 *   sf_swizzle          row-major scale matrix <-> 128x4 swizzled layout
 *   nvfp4_sf_convert_layout  128x4 ("SM100") <-> SM103 scale layout
 *   MoE steps           moe_sort_by_expert, moe_gather_rows, nvfp4_quantize_experts,
 *                       nvfp4_gather_quantize_experts (the two fused),
 *                       nvfp4_silu_mul_quantize_experts, nvfp4_grouped_gemm, moe_combine
 *   nvfp4_gated_gemm    both projections of a feed-forward block, the activation and the product in
 *                       one kernel; nvfp4_gated_gemm_backward: the gradients of both projections
 *   decoder block       block_norm, block_norm_quantize, block_norm_backward (the norms before and
 *                       after a block with its gate and residual sum)
 *   sample_tokens       one token per row of logits: temperature, top-k, top-p, min-p
 *   sizes and status    nvfp4_sf_bytes, mxfp4_grouped_sf_bytes, moe_sort_workspace_size,
 *                       nvfp4_check_status, nvfp4_last_error
 *
 * Sources ("page, section"):
 *   [vLLM-SM103]  vLLM fork compare view "add pdl" (sm103 branch)
 *   [FI-4865]     FlashInfer PR 4865 "perf(gemm): optimize SM103 CuTe DSL mm_fp4 kernel"
 *   [FI-4466]     FlashInfer PR 4466 "sm100 cute_dsl w4a16 gemm" (follow-up PR 4620 text)
 *   [vLLM-51158]  vLLM PR 51158 "Enable CUTLASS MXFP4 W4A4 MoE on SM12x"
 *
 * Conventions shared by every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The library never
 *     allocates device memory (nvfp4_gemm_noalloc's scratch is a static array of the library)
 *     and keeps no pointer after the call returns.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy default stream).
 *   - Arguments are validated on the host before anything is enqueued.  On error nothing
 *     is launched, the status is returned and nvfp4_last_error() describes it.
 *   - Sizes of zero rows are legal and enqueue nothing.
 *   - The current device must be compute capability 10.3 (sm_103).
 *   - Packed FP4: element 2t of a row is the low nibble of byte t, element 2t+1 the high one.
 *   - 128x4 scale layout: a scale matrix of R rows and C scale columns is stored as
 *     round_up(R,128) * round_up(C,4) bytes; scale (r, j) sits at byte
 *       ((r/128) * (round_up(C,4)/4) + j/4) * 512 + (r%32)*16 + ((r/32)%4)*4 + j%4
 *     ([vLLM-SM103] nvfp4_quant_kernels.cu "Scale factor layout conversion: SM100 <-> SM103",
 *     SM100 offset; nvfp4_utils.cuh tile base).  Padding bytes must hold 0x00 (the
 *     quantisers write them so).
 */
#ifndef NVFP4_GB300_H
#define NVFP4_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *nvfp4_stream_t;

typedef enum {
  NVFP4_OK = 0,
  NVFP4_ERR_INVALID_ARG = 1,        /* null pointer, negative size, bad enum value */
  NVFP4_ERR_MISALIGNED = 2,         /* pointer or stride alignment rule broken */
  NVFP4_ERR_UNSUPPORTED_SHAPE = 3,  /* divisibility rule broken (K % 32, N % 32, ...) */
  NVFP4_ERR_UNSUPPORTED_DEVICE = 4, /* current device is not sm_103 */
  NVFP4_ERR_CUDA = 5,               /* a CUDA runtime/driver call failed (message has the name) */
  NVFP4_ERR_TIMEOUT = 6             /* a kernel gave up a bounded wait (nvfp4_check_status) */
} nvfp4_status_t;

/* Launch flags (bitwise OR). */
enum {
  /* Launch with programmatic dependent launch (cudaLaunchAttributeProgrammaticStreamSerialization):
   * the kernel may start while the previous kernel on the stream is still running.  Every
   * kernel of this library waits (griddepcontrol.wait) before it reads an input that a
   * predecessor may produce or writes any output, and signals its own dependents
   * (griddepcontrol.launch_dependents) once its input reads are issued.  Exception, stated
   * per entry point: nvfp4_gemm and mxfp4_grouped_gemm may read the weight operand B and its
   * scales before the wait, so B must not be written by the kernels it overlaps.
   * [vLLM-SM103] summary.md "What is PDL?", nvfp4_quant_kernels.cu "Host entry: SM103
   * activation quantization" (use_pdl). */
  NVFP4_FLAG_PDL = 1u << 0,
  /* Scale buffers in the SM103 layout instead of the 128x4 ("SM100") one: nvfp4_quantize writes
   * its scales, nvfp4_gemm / nvfp4_gemm_noalloc read both sfa and sfb, in that layout.  Same
   * 512-byte tiles in the same order; inside a tile, row m = m4b + 4*m4a + 16*m8 and scale
   * column k sit at m8*16 + m4a*128 + m4b*4 + k.  [vLLM-SM103] nvfp4_quant_kernels.cu "Scale
   * factor layout conversion: SM100 <-> SM103", nvfp4_utils.cuh (SM103 swizzled SF offset).
   * Not accepted by the MXFP4 entry points. */
  NVFP4_FLAG_SF_SM103 = 1u << 2,
  /* Short (about 20 ms) limit on every pipeline wait instead of the default (about 10 s);
   * for tests of the timeout path. */
  NVFP4_FLAG_DEBUG_TIMEOUT = 1u << 8,
  /* Test hook of the time-out path (GEMMs only, honoured only together with
   * NVFP4_FLAG_DEBUG_TIMEOUT): the loader posts the byte count of the first K stage of each CTA
   * but issues none of its copies, so the wait for that stage runs out.  The kernel then records
   * the time-out (nvfp4_check_status returns NVFP4_ERR_TIMEOUT), drains its bounded waits, frees
   * its tensor memory and exits; the output is undefined.  Nothing is read or written out of
   * bounds. */
  NVFP4_FLAG_DEBUG_SKIP_FIRST_LOAD = 1u << 9
};

/* Message for the last error on the calling thread ("" when the last call succeeded). */
const char *nvfp4_last_error(void);

/* Bytes of a swizzled scale buffer for `rows` rows of `k` elements with one scale per
 * `sf_vec` (16 for NVFP4, 32 for MXFP4): round_up(rows,128) * round_up(k/sf_vec, 4).
 * Returns 0 for invalid arguments.  Host only. */
size_t nvfp4_sf_bytes(int64_t rows, int64_t k, int sf_vec);

/* Bytes of the grouped MXFP4 scale buffer that mxfp4_quantize writes for `total_rows` rows
 * split over `num_experts` experts: an upper bound of sum_e round_up(M_e,128) rows, namely
 * (round_up(total_rows,128) + 128*num_experts) * round_up(k/32,4).  Host only. */
size_t mxfp4_grouped_sf_bytes(int64_t total_rows, int num_experts, int64_t k);

/* NVFP4 activation quantisation.
 * Source: [vLLM-SM103] nvfp4_quant_kernels.cu "SM103 (B300) activation quantization kernel"
 * (one fp32 global scale, a scale per 16 elements of a row, packed e2m1 out, swizzled scales,
 * padded scale rows/columns quantised from zero input) and test_nvfp4_quant.py (global scale
 * = 448*6/amax).  Per 16-element block, in fp32 with round-to-nearest-even on every step:
 *   s = (gs*amax)/6; sc = e4m3_satfinite(s); inv = sd ? gs/sd : 0 (sd = value of sc);
 *   q_i = e2m1_satfinite(x_i * inv) (the sign of a zero result is kept).
 *   x        bf16 [m, k], row stride `ldx` elements (ldx >= k, ldx % 8 == 0), 16-B aligned
 *   gs       device fp32 scalar (global scale), 4-B aligned
 *   q        uint8 [m, k/2] row-major, 8-B aligned
 *   sf       uint8 [nvfp4_sf_bytes(m, k, 16)], 16-B aligned; every byte is written
 *   k % 16 == 0.  Reads x/gs and writes q/sf only after the PDL wait. */
nvfp4_status_t nvfp4_quantize(const void *x, int64_t m, int64_t k, int64_t ldx, const float *gs,
                              uint8_t *q, uint8_t *sf, uint32_t flags, nvfp4_stream_t stream);

/* MXFP4 quantisation ("e2m1 data with e8m0 scale per 32", [vLLM-51158] "Changes",
 * mxfp4_experts_quant.cu).  Per 32-element block: s = amax/6 (fp32); scale = smallest power
 * of two >= s (ue8m0 code clamped to [0,254], 0 for an all-zero block);
 * q_i = e2m1_satfinite(x_i * 2^(127-code)).
 *   x            bf16 [t, k], row stride ldx (ldx >= k, ldx % 8 == 0), 16-B aligned
 *   row_offsets  NULL for one dense scale block of round_up(t,128) rows; otherwise a DEVICE
 *                int64 [num_experts+1] array, non-decreasing, row_offsets[0] == 0,
 *                row_offsets[num_experts] == t: rows of expert e are row_offsets[e] ..
 *                row_offsets[e+1]-1 and their scales form their own zero-padded 128-row
 *                block starting at scale row sum_{j<e} round_up(M_j,128).
 *   q            uint8 [t, k/2]; sf uint8 [sf_bytes] (16-B aligned), sf_bytes >=
 *                nvfp4_sf_bytes(t,k,32) (dense) or mxfp4_grouped_sf_bytes(t,E,k) (grouped).
 *   k % 32 == 0, 1 <= num_experts <= 1024 when row_offsets != NULL.
 *   Offsets that break the rules above are a caller error; the kernel never writes outside
 *   q[0..t) rows or sf[0..sf_bytes). */
nvfp4_status_t mxfp4_quantize(const void *x, int64_t t, int64_t k, int64_t ldx,
                              const int64_t *row_offsets, int num_experts, uint8_t *q, uint8_t *sf,
                              size_t sf_bytes, uint32_t flags, nvfp4_stream_t stream);

/* The tile configuration nvfp4_gemm picks for a shape (M-based selector, [vLLM-SM103]
 * nvfp4_scaled_mm_kernels.cu "SM103 Dispatch"; narrow tiles for small M, [FI-4865]
 * "Reviewer Notes").  Up to 256 tokens the weight fills the MMA's 128-row slot and K is split
 * inside clusters, except where 256 x 256 CTA-pair tiles fill a quarter of the pairs, or where K
 * is short (4096 <= N <= 16384 and K <= 2048 from 17 tokens, K <= 4096 from 129): there whole
 * 128 x 128 tiles run.
 * Host only. */
typedef struct {
  int swap_ab;   /* 1: the weight B fills the 128-row MMA slot and tokens the N slot */
  int tile_m;    /* rows of the MMA tile (128) */
  int tile_n;    /* MMA N */
  int splits;    /* K splits reduced inside a thread-block cluster (1 = none) */
  int stages;    /* shared-memory pipeline depth */
  int ctas;      /* CTAs launched */
  int dp_tiles;  /* output tiles each computed whole by one CTA */
  int sk_tiles;  /* output tiles after those whose K stages are split stream-K over all CTAs */
} nvfp4_gemm_plan_t;
nvfp4_status_t nvfp4_gemm_plan(int64_t m, int64_t n, int64_t k, nvfp4_gemm_plan_t *plan);

/* Bytes of device workspace nvfp4_gemm needs for this shape on the current device (0 when the
 * plan splits no tile).  Host only.  The split-K reduction is the library's own design (the
 * pages' kernels pick split-K for small M but do not describe how partials are added): the
 * workspace holds one arrival counter per split tile followed by two fp32 partial-tile slots
 * of 128 x tile_n per CTA. */
nvfp4_status_t nvfp4_gemm_workspace_size(int64_t m, int64_t n, int64_t k, size_t *bytes);

/* NVFP4 block-scaled GEMM with bf16 output.
 * Source: [vLLM-SM103] nvfp4_scaled_mm_kernels.cu "SM103 Entry Point" (A [M,K/2] packed e2m1
 * row-major, B [N,K/2] packed e2m1 K-major, scale_a/scale_b e4m3 in the 128x4 layout padded to
 * [round_up(rows,128), round_up(K/16,4)], alpha fp32 [1], k % 32 == 0, n % 32 == 0);
 * [FI-4865] "2. Alpha epilogue bug" (alpha multiplies the fp32 accumulator, then ONE
 * conversion to bf16) and "3. Restore 256-bit stores" (D compact N-major, 32-B aligned).
 *   D[m,n] = bf16( alpha * sum_k e2m1(A[m,k]) e4m3(sfa[m,k/16]) e2m1(B[n,k]) e4m3(sfb[n,k/16]) )
 *   a      uint8 [m, k/2], 32-B aligned         sfa  nvfp4_sf_bytes(m,k,16) bytes, 16-B aligned
 *   b      uint8 [n, k/2], 32-B aligned         sfb  nvfp4_sf_bytes(n,k,16) bytes, 16-B aligned
 *   alpha  device fp32 scalar, 4-B aligned       d    bf16 [m, n] row-major, 32-B aligned
 *   workspace    device buffer of at least nvfp4_gemm_workspace_size(m,n,k) bytes, 256-B
 *                aligned (may be NULL when that size is 0).  It must be zero-filled before its
 *                first use; every call that completes leaves it zero again, so one zeroing
 *                serves any number of calls.  Calls that can run at the same time (other
 *                streams) need separate workspaces: the kernel's counters and partial tiles
 *                would race.  After a call that reported NVFP4_ERR_TIMEOUT, zero it again.
 *   n % 32 == 0, k % 32 == 0, m, n, k < 2^31.
 * The output does not depend on timing: split tiles are added in a fixed order.
 * With NVFP4_FLAG_PDL, b and sfb may be read before the wait for the preceding kernel; the
 * workspace is touched only after that wait. */
nvfp4_status_t nvfp4_gemm(const uint8_t *a, const uint8_t *sfa, const uint8_t *b, const uint8_t *sfb,
                          const float *alpha, void *d, int64_t m, int64_t n, int64_t k,
                          void *workspace, size_t workspace_bytes, uint32_t flags,
                          nvfp4_stream_t stream);

/* nvfp4_quantize fused into nvfp4_gemm: D = nvfp4_gemm(nvfp4_quantize(x, gs_x), b), with the
 * activation quantised inside the GEMM kernel, so its codes and scales never go through global
 * memory and one launch replaces two.  Not an operation of the pages; it is the "quantise in
 * the GEMM's prologue" extension of [vLLM-SM103] "add pdl" (the PDL edge between the two).
 * The result is bit-identical to the two calls: every 16-element block is quantised with the
 * same arithmetic as nvfp4_quantize and the MMAs consume it in the same order.
 *   x      bf16 [m, k] row-major, row stride ldx >= k elements, 16-B aligned, ldx % 8 == 0
 *   gs_x   device fp32 scalar: x's global scale, as nvfp4_quantize's
 *   b, sfb, alpha, d, workspace, flags, stream: as nvfp4_gemm (NVFP4_FLAG_SF_SM103: sfb is in
 *          the SM103 layout); these plans split K inside clusters and need no workspace.
 *   1 <= m <= 256 (the weight-streaming plans, where each CTA quantises the token rows it
 *   needs; this call takes one for every such m, also where nvfp4_gemm_plan reports another
 *   kind for nvfp4_gemm); larger m: NVFP4_ERR_UNSUPPORTED_SHAPE, nothing launched (quantise
 *   separately).
 *   Every CTA that shares a token tile quantises it again (once per 128 weight rows), so the
 *   fused call is faster than the PDL-chained pair only for a few tokens (measured on GB300,
 *   N=4096, K=7168, cold weights: M=1 3 % faster, M=4 even, M >= 16 slower).
 * With NVFP4_FLAG_PDL, b and sfb may be read before the wait for the preceding kernel; x after it.
 */
nvfp4_status_t nvfp4_quantize_gemm(const void *x, int64_t ldx, const float *gs_x, const uint8_t *b,
                                   const uint8_t *sfb, const float *alpha, void *d, int64_t m, int64_t n,
                                   int64_t k, void *workspace, size_t workspace_bytes, uint32_t flags,
                                   nvfp4_stream_t stream);

/* nvfp4_gemm without a workspace argument: when the plan splits tiles stream-K, the partial
 * tiles and arrival counters go to a static 20 MiB device array inside the library instead of a
 * caller buffer.  The pages have no counterpart of this entry point: it exists for callers that
 * cannot allocate or hold device memory for a workspace at call time, such as a plugin inside an
 * inference engine whose device memory is planned once up front, or code on a latency path where
 * a cudaMalloc would synchronise the device.
 *   Arguments, layouts, alignment and errors are those of nvfp4_gemm.  The call never allocates.
 *   Shapes whose workspace (nvfp4_gemm_workspace_size) exceeds the array (20 MiB + 4 KiB) are
 *   refused with NVFP4_ERR_UNSUPPORTED_SHAPE; every plan the selector makes on a GPU of up to
 *   160 SMs fits (the largest: 80 split tiles on 160 CTAs, 20 MiB + 512 bytes).
 *   The array is shared by every call on the device: calls that may overlap (other streams,
 *   other threads) race on it and must not use this entry point concurrently.
 *   The array's address is looked up (cudaGetSymbolAddress) on the first call on each device,
 *   and again on the first call after the device got a new context (a device reset); a caller
 *   that records work for later replay should make one call before it starts recording.
 *   The arrival counters must read zero when the kernel starts: before each launch of a split
 *   plan this entry point enqueues a one-CTA kernel on `stream` that clears them (so a call
 *   after one that timed out starts clean); the partial-tile slots need no initialisation.
 *   That kernel takes the call's NVFP4_FLAG_PDL too: it waits for the preceding kernel before
 *   clearing, while the GEMM starts beside it and streams its weight as nvfp4_gemm would. */
nvfp4_status_t nvfp4_gemm_noalloc(const uint8_t *a, const uint8_t *sfa, const uint8_t *b, const uint8_t *sfb,
                                  const float *alpha, void *d, int64_t m, int64_t n, int64_t k,
                                  uint32_t flags, nvfp4_stream_t stream);

/* Gated product of a feed-forward block: both projections, the activation and the product in one
 * kernel, bf16 out.
 *   h[t, j] = bf16( act(alpha[0] * sum_k A[t,k] Bg[j,k]) * (alpha[1] * sum_k A[t,k] Bu[j,k]) )
 * with A, Bg and Bu the dequantised operands, fp32 sums, and act
 *   NVFP4_ACT_SILU       g / (1 + exp(-g))
 *   NVFP4_ACT_GELU_TANH  g/2 * (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3)))
 * (fp32; approximate exponential and reciprocal: 1 / (1 + exp(-q)) is within 2^-15 of itself, and 0 where
 * exp(-q) passes 2^126; one rounding, at the end).  NaN products give NaN in h and in every gradient they enter.
 * The pages fuse the activation with the quantiser after the product ([vLLM-SM103] ops.h,
 * silu_and_mul_scaled_fp4_experts_quant); here it is the product's epilogue, so the [m, 2 inter]
 * pre-activations never reach memory.
 *   a, sfa   as nvfp4_gemm
 *   b, sfb   uint8 [2*inter, k/2] and its scales (of 2*inter rows): the gate and the up weight in one
 *            matrix whose rows alternate in groups of 16, gate rows first: row 32 j + i is gate row
 *            16 j + i and row 32 j + 16 + i is up row 16 j + i, for i < 16.  Laid out once, when the
 *            weight is quantised.
 *   alpha    device fp32 [2]: the factor of the gate and of the up product, 4-B aligned
 *   h        bf16 [m, inter] row-major, 32-B aligned
 *   workspace, flags, stream: as nvfp4_gemm with n = 2*inter (nvfp4_gemm_workspace_size(m, 2*inter, k))
 *   inter % 16 == 0, k % 32 == 0.  PDL and reproducibility as nvfp4_gemm. */
enum { NVFP4_ACT_SILU = 0, NVFP4_ACT_GELU_TANH = 1 };
nvfp4_status_t nvfp4_gated_gemm(const uint8_t *a, const uint8_t *sfa, const uint8_t *b, const uint8_t *sfb,
                                const float *alpha, int activation, void *h, int64_t m, int64_t inter, int64_t k,
                                void *workspace, size_t workspace_bytes, uint32_t flags, nvfp4_stream_t stream);

/* Backward pass of nvfp4_gated_gemm up to its two products: with g and u the products (computed again
 * from the packed operands, so the forward pass stores nothing),
 *   dgu[t, 32 j + i]      = bf16(dh[t, 16 j + i] * u * act'(g))       gradient of the gate product
 *   dgu[t, 32 j + 16 + i] = bf16(dh[t, 16 j + i] * act(g))            gradient of the up product
 * in the row order of b, so that the gradient of the input is dgu B and that of the weight dgu^T A:
 * products that nvfp4_quantize and nvfp4_gemm compute from the transposed operands.
 *   dh   bf16 [m, inter], 32-B aligned;  dgu  bf16 [m, 2*inter], 32-B aligned
 *   h    bf16 [m, inter], 32-B aligned, or NULL: the forward result, which the gradient of the next
 *        weight needs
 * Everything else as nvfp4_gated_gemm. */
nvfp4_status_t nvfp4_gated_gemm_backward(const uint8_t *a, const uint8_t *sfa, const uint8_t *b, const uint8_t *sfb,
                                         const float *alpha, int activation, const void *dh, void *dgu, void *h,
                                         int64_t m, int64_t inter, int64_t k, void *workspace, size_t workspace_bytes,
                                         uint32_t flags, nvfp4_stream_t stream);

/* MXFP4 grouped (MoE) GEMM: for every expert e, D[rows of e, :] = alpha * deq(A_e) deq(B_e)^T.
 * The kernel checks row_offsets on the device (row_offsets[0] == 0, row_offsets[E] == t,
 * non-decreasing); if they are malformed it does no work and nvfp4_check_status reports
 * NVFP4_ERR_INVALID_ARG.
 * Source: [vLLM-51158] "Changes" (CUTLASS MXFP4 grouped GEMM over experts; SM10x/SM12x share
 * the block-scaled scale layout) and [vLLM-SM103] ops.h (expert offsets as arguments).
 *   a            uint8 [t, k/2] (rows sorted by expert), 32-B aligned
 *   sfa          grouped ue8m0 scales as mxfp4_quantize(row_offsets) writes them, 16-B aligned
 *   row_offsets  DEVICE int64 [num_experts+1] (same rules as mxfp4_quantize)
 *   b            uint8 [num_experts, n, k/2], 32-B aligned
 *   sfb          uint8 [num_experts, nvfp4_sf_bytes(n,k,32)] (each expert's block swizzled)
 *   alpha        device fp32 scalar or NULL for 1.0
 *   d            bf16 [t, n] row-major, 32-B aligned
 *   n % 32 == 0, k % 32 == 0, 1 <= num_experts <= 1024.
 * With NVFP4_FLAG_PDL, b and sfb may be read before the wait for the preceding kernel. */
nvfp4_status_t mxfp4_grouped_gemm(const uint8_t *a, const uint8_t *sfa, const int64_t *row_offsets,
                                  int num_experts, const uint8_t *b, const uint8_t *sfb,
                                  const float *alpha, void *d, int64_t t, int64_t n, int64_t k,
                                  uint32_t flags, nvfp4_stream_t stream);

/* ---------------------------------------------------------------- MoE steps (NVFP4)
 * The steps around the grouped GEMMs of an NVFP4 mixture-of-experts layer:
 *   moe_sort_by_expert -> moe_gather_rows -> nvfp4_quantize_experts -> nvfp4_grouped_gemm (gate+up)
 *   -> nvfp4_silu_mul_quantize_experts -> nvfp4_grouped_gemm (down) -> moe_combine.
 * [vLLM-SM103] ops.h / torch_bindings.cpp name scaled_fp4_experts_quant,
 * silu_and_mul_scaled_fp4_experts_quant (arguments input_offset_by_experts,
 * output_scale_offset_by_experts) and cutlass_fp4_group_mm; [vLLM-51158] "Changes" describes the
 * experts-quantise + grouped-GEMM structure.  The pages give names and arguments only; the
 * definitions below are this library's reading of them. */

/* Bytes of device workspace moe_sort_by_expert needs (one int32 count per CTA and expert).  Host only. */
size_t moe_sort_workspace_size(int64_t num_tokens, int num_experts);

/* Stable sort of routed (token, slot) pairs by expert.
 *   topk_ids     DEVICE int32 [num_tokens, topk], expert of each slot (0 <= id < num_experts;
 *                other values are dropped (pos = -1) and make nvfp4_check_status report
 *                NVFP4_ERR_INVALID_ARG)
 *   row_offsets  DEVICE int64 [num_experts + 1] out: rows of expert e are row_offsets[e] ..
 *                row_offsets[e+1]-1 of the permuted order (the grouped kernels' row_offsets)
 *   src_rows     DEVICE int32 [num_tokens * topk] out: token of each permuted row
 *   pos          DEVICE int32 [num_tokens, topk] out: permuted row of each (token, slot)
 *   workspace    DEVICE, 4-B aligned, workspace_bytes >= moe_sort_workspace_size(); no
 *                initialisation needed (every byte used is written first)
 * Inside an expert, rows keep (token, slot) row-major order.  1 <= topk <= 32,
 * 1 <= num_experts <= 1024, num_tokens * topk <= 2^31 - 512.  Two kernels over ceil(num_tokens/32) CTAs (at most 1024). */
nvfp4_status_t moe_sort_by_expert(const int32_t *topk_ids, int64_t num_tokens, int topk, int num_experts,
                                  int64_t *row_offsets, int32_t *src_rows, int32_t *pos, int32_t *workspace,
                                  size_t workspace_bytes, uint32_t flags, nvfp4_stream_t stream);

/* Row gather (permutation into expert order): out[r, :] = x[src_rows[r], :] for r < rows.
 *   x        bf16 [num_tokens, h], row stride ldx (ldx >= h, ldx % 8 == 0), 16-B aligned
 *   out      bf16 [rows, h] contiguous, 16-B aligned; h % 8 == 0
 * A src_rows entry outside [0, num_tokens) is skipped (that row is not written) and makes
 * nvfp4_check_status report NVFP4_ERR_INVALID_ARG. */
nvfp4_status_t moe_gather_rows(const void *x, int64_t num_tokens, int64_t h, int64_t ldx, const int32_t *src_rows,
                               int64_t rows, void *out, uint32_t flags, nvfp4_stream_t stream);

/* Per-expert NVFP4 quantisation (scaled_fp4_experts_quant): rows of expert e (row_offsets as
 * moe_sort_by_expert writes them) are quantised as nvfp4_quantize does with global scale gs[e];
 * expert e's scales form their own zero-padded 128-row block starting at scale row
 * sum_{j<e} round_up(M_j, 128) of a round_up(k/16, 4)-column 128x4-swizzled matrix.
 *   x      bf16 [t, k], row stride ldx, 16-B aligned;  gs  DEVICE fp32 [num_experts]
 *   q      uint8 [t, k/2], 8-B aligned
 *   sf     uint8 [sf_bytes], 16-B aligned, sf_bytes >= (round_up(t,128) + 128*num_experts) *
 *          round_up(k/16, 4)  (the same bound as mxfp4_grouped_sf_bytes with k/16 columns)
 *   k % 16 == 0, 1 <= num_experts <= 1024. */
nvfp4_status_t nvfp4_quantize_experts(const void *x, int64_t t, int64_t k, int64_t ldx, const int64_t *row_offsets,
                                      int num_experts, const float *gs, uint8_t *q, uint8_t *sf, size_t sf_bytes,
                                      uint32_t flags, nvfp4_stream_t stream);

/* moe_gather_rows fused into nvfp4_quantize_experts: row r of the quantised matrix is row
 * src_rows[r] of x, so the gathered bf16 copy is never written.  For src_rows entries in
 * [0, num_tokens) the result (q, sf) is bit-identical to moe_gather_rows(x, src_rows) followed
 * by nvfp4_quantize_experts on its output.  A row whose entry is outside [0, num_tokens) is
 * quantised from zeros and makes nvfp4_check_status report NVFP4_ERR_INVALID_ARG.  The sources
 * define no such call: it joins two of the steps above ([vLLM-SM103] ops.h quantises the
 * already permuted activation with scaled_fp4_experts_quant).
 *   x         bf16 [num_tokens, k], row stride ldx >= k (ldx % 8 == 0), 16-B aligned
 *   src_rows  DEVICE int32 [rows] (as moe_sort_by_expert writes it), 4-B aligned
 *   row_offsets, num_experts, gs, q ([rows, k/2]), sf, sf_bytes: as nvfp4_quantize_experts
 *   with t = rows.  (rows + 128*num_experts) * round_up(k/16,4) < 2^31, else
 *   NVFP4_ERR_UNSUPPORTED_SHAPE (quantise the gathered rows with nvfp4_quantize_experts). */
nvfp4_status_t nvfp4_gather_quantize_experts(const void *x, int64_t num_tokens, int64_t k, int64_t ldx,
                                             const int32_t *src_rows, int64_t rows, const int64_t *row_offsets,
                                             int num_experts, const float *gs, uint8_t *q, uint8_t *sf,
                                             size_t sf_bytes, uint32_t flags, nvfp4_stream_t stream);

/* SiLU-and-mul fused with the per-expert NVFP4 quantisation (silu_and_mul_scaled_fp4_experts_quant).
 * x is bf16 [t, 2*inter] = [gate | up]; the quantised matrix is h [t, inter] with
 *   h = bf16(silu(gate) * up),  silu(g) = g * (1 / (1 + exp(-g)))  in fp32,
 * exp computed by Cody-Waite range reduction and a degree-7 Taylor polynomial, every fp32 step
 * rounded to nearest even (so the result equals "silu_and_mul to bf16, then quantise" done the
 * same way), then h is quantised as nvfp4_quantize_experts does (q [t, inter/2], sf as there
 * with k = inter).  ldx >= 2*inter, inter % 16 == 0. */
nvfp4_status_t nvfp4_silu_mul_quantize_experts(const void *x, int64_t t, int64_t inter, int64_t ldx,
                                               const int64_t *row_offsets, int num_experts, const float *gs,
                                               uint8_t *q, uint8_t *sf, size_t sf_bytes, uint32_t flags,
                                               nvfp4_stream_t stream);

/* NVFP4 grouped (MoE) GEMM (cutlass_fp4_group_mm): D[rows of e, :] = alpha[e] * deq(A_e) deq(B_e)^T.
 *   a      uint8 [t, k/2] rows sorted by expert;  sfa  as nvfp4_quantize_experts writes it
 *   b      uint8 [num_experts, n, k/2];  sfb  uint8 [num_experts, nvfp4_sf_bytes(n, k, 16)]
 *   alpha  DEVICE fp32 [num_experts] (one per expert: 1/(gsA_e * gsB_e)) or NULL for 1.0
 *   d      bf16 [t, n], 32-B aligned;  n % 32 == 0, k % 32 == 0;  1 <= num_experts <= 512 (the
 *          expert tables share the CTA's shared memory with the operand ring: 128 x 256 tiles on a
 *          4-deep ring up to 256 experts, 128 x 128 tiles beyond).
 * Same kernel, other checks and PDL behaviour as mxfp4_grouped_gemm. */
nvfp4_status_t nvfp4_grouped_gemm(const uint8_t *a, const uint8_t *sfa, const int64_t *row_offsets, int num_experts,
                                  const uint8_t *b, const uint8_t *sfb, const float *alpha, void *d, int64_t t,
                                  int64_t n, int64_t k, uint32_t flags, nvfp4_stream_t stream);

/* Weighted combine of the experts' outputs:
 *   out[t, :] = bf16( sum_{j < topk} weights[t, j] * y[pos[t, j], :] )
 * in fp32, slots in order, each product and sum rounded (no fused multiply-add); slots with
 * pos < 0 are skipped (a token with none gets zeros); pos >= rows is skipped too and makes
 * nvfp4_check_status report NVFP4_ERR_INVALID_ARG.
 *   y        bf16 [rows, h] (expert order), 16-B aligned;  pos  DEVICE int32 [num_tokens, topk]
 *   weights  DEVICE fp32 [num_tokens, topk];  out  bf16 [num_tokens, h], 16-B aligned;  h % 8 == 0 */
nvfp4_status_t moe_combine(const void *y, int64_t rows, const int32_t *pos, const float *weights,
                           int64_t num_tokens, int topk, int64_t h, void *out, uint32_t flags,
                           nvfp4_stream_t stream);

/* ---------------------------------------------------------------- norms around a decoder block
 * The RMS norm after a block, the block's gate, the residual sum and the norm before the next
 * block, in one pass over the rows.  For a row of n channels, in fp32:
 *   p = y * rsqrt(mean(y^2) + eps) * (weight_offset + w_post)    (p = y when w_post is NULL)
 *   r = x + residual_scale * (gate * p)                          (gate = 1 when NULL; r = x when y is NULL)
 *   h = r * rsqrt(mean(r^2) + eps) * (weight_offset + w_pre)
 * r is rounded once, to x's type, when it is stored in x_out; h is computed from the unrounded r
 * and rounded once, to bf16.  Not operations of the pages: they are what a decoder runs between
 * the products of this library.  weight_offset is 1 for weights stored around zero, else 0.
 *   x       bf16 or fp32 (x_type: NVFP4_DTYPE_*) [m, n], row stride ldx elements
 *   y       bf16 [m, n], row stride ldy; NULL: no block before this norm (then w_post, gate and
 *           x_out are NULL too)
 *   w_post, w_pre   bf16 [n]; w_pre and h may both be NULL (no norm after the sum)
 *   gate    bf16 [m, n] with row stride ldg, or [n] shared by all rows with ldg = 0
 *   x_out   x's type [m, n], row stride ldxo; may be x itself (same stride); no other overlap
 *   h       bf16 [m, n], row stride ldh
 *   1 <= n <= 32768.  Any strides (of an input also 0: one row for all) and alignments of whole
 *   elements are taken; rows that all start on 16 bytes (and n % 8 == 0) are moved with 16-byte accesses.
 * Every input is read and every output written after the PDL wait. */
enum { NVFP4_DTYPE_BF16 = 0, NVFP4_DTYPE_F32 = 1 };
nvfp4_status_t block_norm(const void *x, int x_type, int64_t ldx, const void *y, int64_t ldy, const void *w_post,
                          const void *gate, int64_t ldg, const void *w_pre, float residual_scale, float eps,
                          float weight_offset, void *x_out, int64_t ldxo, void *h, int64_t ldh, int64_t m, int64_t n,
                          uint32_t flags, nvfp4_stream_t stream);

/* block_norm whose h goes out as NVFP4, ready for nvfp4_gemm: q and sf equal nvfp4_quantize of
 * block_norm's h under global scale gs, bit for bit, for an h whose rows start on 16 bytes too (other rows
 * are computed with their sums in another order); scale rows up to the next multiple of 128 are
 * zeroed.  n % 16 == 0; every row of x, y, gate and x_out, the weights and sf on 16 bytes. */
nvfp4_status_t block_norm_quantize(const void *x, int x_type, int64_t ldx, const void *y, int64_t ldy,
                                   const void *w_post, const void *gate, int64_t ldg, const void *w_pre,
                                   float residual_scale, float eps, float weight_offset, void *x_out, int64_t ldxo,
                                   const float *gs, uint8_t *q, uint8_t *sf, int64_t m, int64_t n, uint32_t flags,
                                   nvfp4_stream_t stream);

/* Backward pass of block_norm, from what the forward pass stored.  dh is the gradient of h, dx_out
 * the gradient that reaches x_out from elsewhere (NULL: zero), x_out the stored stream (x itself
 * when y was NULL).
 *   dx       x's type [m, n]: gradient of x, which is also the whole gradient of x_out
 *   dy       bf16 [m, n]
 *   dw_pre, dw_post   fp32 [n], summed over the rows in a fixed order (bit-reproducible)
 *   dgate    bf16 [m, n] (row stride lddg) for a gate per token, fp32 [n] for a gate per channel
 *   dh and w_pre may both be NULL (h was not computed); a NULL w_post or gate has no gradient.
 *   dx may be dx_out and dy may be y (same strides); no other overlap.
 *   workspace   device, 16-B aligned, at least block_norm_backward_workspace_size(m, n) bytes (the
 *               teams' column sums; no initialisation); may be NULL when nothing is summed over rows.
 *               Calls that may overlap need separate ones.
 * Two launches (one when nothing is summed over rows).  m = 0 writes zero to the row sums. */
size_t block_norm_backward_workspace_size(int64_t m, int64_t n);
nvfp4_status_t block_norm_backward(const void *dh, int64_t lddh, const void *dx_out, int64_t lddxo, const void *x_out,
                                   int x_type, int64_t ldxo, const void *y, int64_t ldy, const void *w_post,
                                   const void *gate, int64_t ldg, const void *w_pre, float residual_scale, float eps,
                                   float weight_offset, void *dx, int64_t lddx, void *dy, int64_t lddy, float *dw_pre,
                                   float *dw_post, void *dgate, int64_t lddg, int64_t m, int64_t n, void *workspace,
                                   size_t workspace_bytes, uint32_t flags, nvfp4_stream_t stream);

/* ---------------------------------------------------------------- draw of the next token
 * One token per row of logits, from a random number given per row.  Not an operation of the pages:
 * it is what a decoder does with the last product's rows.  For a row z with largest logit m (fp32,
 * each step rounded to nearest):
 *   x_i = (z_i - m) * (log2(e) / temperature),  e_i = 2^x_i,  w_i = rint(e_i * 2^30)
 * (2^x by the hardware's approximation, within 2^-22).  Tokens are ordered by x, largest first, ties by
 * index; each filter keeps a beginning of that order, and the first token always stays:
 *   top_k   the first top_k (<= 0: all)
 *   top_p   those before which the top_k weigh less than top_p * their total (>= 1 or NaN: all)
 *   min_p   those with e_i >= min_p (<= 0: all; above 1 or NaN: none but the first token)
 * The token is the first, by index, at which the kept tokens' cumulative weight exceeds
 * floor(uniform * total).  The weights are whole numbers and their sums exact, so the result depends
 * neither on timing nor on how a row is split.
 *   logits       bf16 or fp32 (logits_type: NVFP4_DTYPE_*) [rows, vocab], row stride ld >= vocab or
 *                0 (one row for all), any alignment of whole elements.  NaN and -inf weigh nothing;
 *                with +inf only the +inf tokens weigh.  A row with nothing else than NaN and -inf gives token -1.
 *   uniform      fp32 [rows], in [0, 1) (values outside draw the first or the last kept token)
 *   temperature  fp32 [rows] or NULL for 1; <= 0 (or NaN): the largest logit, lowest index
 *   top_k        int32 [rows] or NULL;  top_p, min_p  fp32 [rows] or NULL
 *   tokens       int32 [rows]
 *   logprobs     fp32 [rows] or NULL: log of the token's probability among the kept ones (-inf for
 *                token -1)
 *   1 <= vocab <= 2^21, rows < 2^28.  One launch, no workspace.
 * Every input is read and every output written after the PDL wait. */
nvfp4_status_t sample_tokens(const void *logits, int logits_type, int64_t ld, const float *uniform,
                             const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                             int32_t *tokens, float *logprobs, int64_t rows, int64_t vocab, uint32_t flags,
                             nvfp4_stream_t stream);

/* ---- 8-bit products scaled per block of 128, and what an expert layer trains with ----
 *
 * e4m3 quantisation with one fp32 scale per block of 128.  A block whose largest magnitude is amax
 * (taken as at least 2^-100) gets
 *   s = fl(amax / 448),  codes e4m3(fl(x * fl(448 / amax)))  (RNE, saturating)
 * with fl one rounding to fp32, so that a code times s stands for x within 2^-4 of x where |x| is
 * at least amax * 2^-6 / 448, and within amax / 448 * 2^-10 below (each but for the fp32 roundings).  A block that holds an infinity or a NaN
 * comes back as no finite number.  The sources quantise to 4 bits only; this is the 8-bit counterpart
 * of nvfp4_quantize, with blocks of the usual 128.
 *   x           bf16 or fp32 (x_type: NVFP4_DTYPE_*) [x_rows, k], row stride ldx >= k or 0 (one row for all);
 *               k % 16 == 0,
 *               every row starts on 16 bytes
 *   src_rows    int32 [rows] or NULL: row r of the result is row src_rows[r] of x (without it rows ==
 *               x_rows).  An entry outside [0, x_rows) quantises zeros and makes nvfp4_check_status
 *               report NVFP4_ERR_INVALID_ARG (x itself must not be NULL where rows > 0).
 *   q, sf       along the rows: e4m3 [rows, k], fp32 [ceil(k/128), rows]: one scale per row and
 *               128 columns (a block of columns' scales lie together), or both NULL
 *   qt, sft     along the columns, transposed: e4m3 [k, P], fp32 [P/128, k] with
 *               P = fp8_padded_rows(rows, num_experts): one scale per column and 128 rows, or both NULL.
 *               Columns past the last row hold zeros (as codes of their block: beside a NaN they stand for NaN).
 *   row_offsets int64 [num_experts+1] on the device (as moe_sort_by_expert writes it; its last entry
 *               may be below rows) or NULL with num_experts 0.  Expert e's rows begin at column
 *               sum_{j<e} round_up(M_j, 128) of qt, so that no block spans two experts; rows past the last
 *               expert's are not quantised (q and sf stay as they were there).  Needs qt.  Malformed
 *               offsets: the columns of qt are zeros and nvfp4_check_status reports
 *               NVFP4_ERR_INVALID_ARG.
 *   q and qt 16-B aligned; 1 <= num_experts <= 1024; rows <= 2^31 - 512, k <= 65535 * 128.
 * x is read once for both. */
int64_t fp8_padded_rows(int64_t rows, int num_experts); /* round_up(rows, 128) + 128 * num_experts */
nvfp4_status_t fp8_quantize(const void *x, int x_type, int64_t x_rows, int64_t k, int64_t ldx, const int32_t *src_rows,
                            int64_t rows, const int64_t *row_offsets, int num_experts, uint8_t *q, float *sf, uint8_t *qt,
                            float *sft, uint32_t flags, nvfp4_stream_t stream);

/* The same for weights, one scale per 128 x 128 block.
 *   w       bf16 or fp32 [matrices, n, k], row stride ldw (matrix stride n * ldw), k % 16 == 0,
 *           every row starts on 16 bytes
 *   q, sf   e4m3 [matrices, n, k], fp32 [matrices, ceil(n/128), ceil(k/128)]
 *   qt, sft the transposes, e4m3 [matrices, k, n] and fp32 [matrices, ceil(k/128), ceil(n/128)]: the same
 *           codes and scales, for the gradient of the product's input; or both NULL.  n % 16 == 0 with them. */
nvfp4_status_t fp8_quantize_weight(const void *w, int w_type, int64_t matrices, int64_t n, int64_t k, int64_t ldw, uint8_t *q,
                                   float *sf, uint8_t *qt, float *sft, uint32_t flags, nvfp4_stream_t stream);

/* Product of two such matrices:
 *   D[i, j] = sum over blocks b of sa[i, b] * sb[j, b] * (sum over the block's k of A[i, k] B[j, k])
 * The sums inside a block are the tensor core's, the scaled sums over the blocks fp32; one rounding to
 * D's type at the end.  The order of the two scales is the kernel's, but over all scales that the quantiser gives (2^-109
 * to 2^120) a block's term leaves fp32's range only where sa * sb * its sum does.
 *   a, sfa   e4m3 [m, k] and fp32 [ceil(k/128), m], as fp8_quantize's q and sf
 *   b, sfb   e4m3 [n, k]; block_b = 128: fp32 [ceil(n/128), ceil(k/128)] (fp8_quantize_weight);
 *            block_b = 1: fp32 [ceil(k/128), n] (fp8_quantize)
 *   d        bf16 or fp32 (d_type) [m, n];  accumulate != 0: D is added to (fp32 only)
 *   a, b and d 16-B aligned, the scales 4-B; k % 16 == 0, any m (0: nothing is done) and any n >= 1.
 * Gradients with the same call: of the input, fp8_gemm(dY, W^T) with W's qt and sft; of the weight,
 * fp8_gemm(dY^T, X^T) with block_b = 1 and both operands from qt and sft.
 * Every operand is read after the PDL wait.  Results do not depend on timing.  No workspace. */
nvfp4_status_t fp8_gemm(const uint8_t *a, const float *sfa, const uint8_t *b, const float *sfb, int block_b, void *d,
                        int d_type, int accumulate, int64_t m, int64_t n, int64_t k, uint32_t flags, nvfp4_stream_t stream);

/* The product of every expert's rows with its weight: D[rows of e, :] = A_e B_e^T, scaled as fp8_gemm with
 * block_b = 128.
 *   a, sfa       e4m3 [t, k] (rows sorted by expert), fp32 [ceil(k/128), t]
 *   row_offsets  DEVICE int64 [num_experts+1]: 0 first, non-decreasing, the last at most t.  Rows of D past
 *                the last expert's stay as they were.  Malformed offsets: no work, and
 *                nvfp4_check_status reports NVFP4_ERR_INVALID_ARG.
 *   b, sfb       e4m3 [num_experts, n, k], fp32 [num_experts, ceil(n/128), ceil(k/128)]
 *   d            bf16 or fp32 [t, n]
 * 1 <= num_experts <= 1024, num_experts * n < 2^31; otherwise as fp8_gemm. */
nvfp4_status_t fp8_grouped_gemm(const uint8_t *a, const float *sfa, const int64_t *row_offsets, int num_experts,
                                const uint8_t *b, const float *sfb, void *d, int d_type, int64_t t, int64_t n, int64_t k,
                                uint32_t flags, nvfp4_stream_t stream);

/* The gradient of every expert's weight: D[e] = A_e^T B_e over the expert's rows, with A the gradient of
 * the product's output and B its input, both as fp8_quantize's qt and sft under the same row_offsets:
 *   a, sfa       e4m3 [n, P], fp32 [P/128, n];  b, sfb  e4m3 [k, P], fp32 [P/128, k]
 *   padded_rows  P, a multiple of 128 with room for every expert's padded rows (fp8_padded_rows)
 *   d            bf16 or fp32 (d_type) [num_experts, n, k];  accumulate != 0: D is added to (fp32 only).
 *                An expert without rows gets zeros (with accumulate: stays).
 * any n (0: nothing is done) and any k >= 1; otherwise as fp8_grouped_gemm. */
nvfp4_status_t fp8_grouped_weight_grad(const uint8_t *a, const float *sfa, const uint8_t *b, const float *sfb,
                                       const int64_t *row_offsets, int num_experts, void *d, int d_type, int accumulate,
                                       int64_t padded_rows, int64_t n, int64_t k, uint32_t flags, nvfp4_stream_t stream);

/* Backward pass of moe_combine: with dout the gradient of its result,
 *   dy[pos[t, j], :]  = bf16(weights[t, j] * dout[t, :])
 *   dweights[t, j]    = sum_c dout[t, c] * y[pos[t, j], c]     (fp32; 0 where pos[t, j] < 0)
 *   dout  bf16 [num_tokens, h], row stride ldo >= h or 0 (one row for all), ldo % 8 == 0;  y, dy  bf16 [rows, h];  16-B aligned, h % 8 == 0
 *   pos   int32 [num_tokens, topk], as moe_sort_by_expert writes it: no row twice (the rows of dy that are named
 *         are each written by their slot, the others stay as they were).  An entry >= rows is skipped as
 *         one < 0 is, and makes nvfp4_check_status report NVFP4_ERR_INVALID_ARG.
 *   Inputs and outputs must not overlap. */
nvfp4_status_t moe_combine_backward(const void *dout, int64_t ldo, const void *y, int64_t rows, const int32_t *pos,
                                    const float *weights, int64_t num_tokens, int topk, int64_t h, void *dy, float *dweights,
                                    uint32_t flags, nvfp4_stream_t stream);

/* Backward pass of moe_gather_rows under moe_sort_by_expert's src_rows: dx[t, :] = bf16(sum_j dxs[pos[t, j], :])
 * in fp32, slots in order.
 *   dxs  bf16 [rows, h], the gradient of the gathered rows;  dx  bf16 [num_tokens, h];  16-B aligned, h % 8 == 0
 *   pos  as above (entries < 0 add nothing; a row may be named more than once). */
nvfp4_status_t moe_gather_backward(const void *dxs, int64_t rows, const int32_t *pos, int64_t num_tokens, int topk, int64_t h,
                                   void *dx, uint32_t flags, nvfp4_stream_t stream);

/* Scale layout conversion between a row-major scale matrix [rows, cols] (bytes) and the
 * 128x4 swizzled layout of nvfp4_sf_bytes size (swizzle writes the zero padding).
 * Source: [vLLM-SM103] nvfp4_utils.py swizzle_blockscale (pad to (128,4), then block
 * interleave) and the in-tile offset quoted at the top of this header.
 *   to_swizzled = 1: src [rows, cols] row-major -> dst swizzled
 *   to_swizzled = 0: src swizzled -> dst [rows, cols] row-major
 * Buffers must not overlap.  No alignment requirement. */
nvfp4_status_t sf_swizzle(const uint8_t *src, uint8_t *dst, int64_t rows, int64_t cols,
                          int to_swizzled, nvfp4_stream_t stream);

/* Converts a swizzled NVFP4 scale buffer between the 128x4 ("SM100") layout and the SM103
 * layout (see NVFP4_FLAG_SF_SM103): every byte of every 512-byte tile moves to its place in the
 * other layout, padding bytes included.
 * Source: [vLLM-SM103] nvfp4_quant_kernels.cu "Scale factor layout conversion: SM100 <-> SM103"
 * (convert_sf_layout_sm100_to_sm103 / _sm103_to_sm100).
 *   src, dst   uint8 [round_up(rows,128) * round_up(cols,4)], 16-B aligned, must not overlap
 *   rows, cols the scale matrix (cols = K/16 scale columns)
 *   to_sm103   1: SM100 -> SM103, 0: SM103 -> SM100
 * Reads src only after the PDL wait (NVFP4_FLAG_PDL semantics are implied: the kernel always
 * waits, so it is safe after any producer). */
nvfp4_status_t nvfp4_sf_convert_layout(const uint8_t *src, uint8_t *dst, int64_t rows, int64_t cols,
                                       int to_sm103, nvfp4_stream_t stream);

/* Synchronises `stream`, then reads and clears the device status word that kernels set when a
 * bounded pipeline wait gave up, a grouped GEMM found malformed row offsets or a MoE step found
 * an index out of range.  Returns NVFP4_ERR_INVALID_ARG for malformed offsets or indices, NVFP4_ERR_TIMEOUT if a
 * kernel timed out since the last check, NVFP4_ERR_CUDA if the synchronisation failed,
 * NVFP4_OK otherwise.
 * The word is one per device, shared by every stream and thread: the call reports what any of
 * this library's kernels on the current device recorded since the previous check, and a bit
 * that a kernel on another, still-running stream sets between the read and the clear is lost.
 * For an exact account, call it when no other stream of the device has this library's work in
 * flight. */
nvfp4_status_t nvfp4_check_status(nvfp4_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_GB300_H */
