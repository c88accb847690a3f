// Entry points of the plain dense NVFP4 GEMM (selector and launch: dense.cuh; kernel: gemm.cuh).
#include "dense.cuh"

using namespace nvfp4;

extern "C" nvfp4_status_t nvfp4_gemm_plan(int64_t m, int64_t n, int64_t k, nvfp4_gemm_plan_t *plan) {
  clear_error();
  if (!plan || m < 0 || n <= 0 || k <= 0) return fail(NVFP4_ERR_INVALID_ARG, "nvfp4_gemm_plan: bad arguments");
  const Plan pl = select_plan(m, n, k, plan_sm_count());
  plan->swap_ab = pl.swap;
  plan->tile_m = pl.pair ? 256 : 128;
  plan->tile_n = pl.bn;
  plan->splits = pl.splits;
  plan->stages = pl.stages;
  plan->ctas = pl.ctas;
  plan->dp_tiles = pl.dp_tiles;
  plan->sk_tiles = pl.sk_tiles;
  return NVFP4_OK;
}

extern "C" nvfp4_status_t nvfp4_gemm_workspace_size(int64_t m, int64_t n, int64_t k, size_t *bytes) {
  clear_error();
  if (!bytes || m < 0 || n <= 0 || k <= 0) return fail(NVFP4_ERR_INVALID_ARG, "nvfp4_gemm_workspace_size: bad arguments");
  *bytes = m == 0 ? 0 : select_plan(m, n, k, plan_sm_count()).ws_bytes;
  return NVFP4_OK;
}

extern "C" nvfp4_status_t nvfp4_gemm(const uint8_t *a, const uint8_t *sfa, const uint8_t *b,
                                     const uint8_t *sfb, const float *alpha, void *d, int64_t m,
                                     int64_t n, int64_t k, void *workspace, size_t workspace_bytes,
                                     uint32_t flags, nvfp4_stream_t stream) {
  clear_error();
  return run_gemm("nvfp4_gemm", a, sfa, b, sfb, alpha, d, m, n, k, workspace, workspace_bytes, flags, stream,
                  FusedA{nullptr, 0, nullptr});
}

extern "C" nvfp4_status_t nvfp4_quantize_gemm(const void *x, int64_t ldx, const float *gs_x, const uint8_t *b,
                                              const uint8_t *sfb, const float *alpha, void *d, int64_t m,
                                              int64_t n, int64_t k, void *workspace, size_t workspace_bytes,
                                              uint32_t flags, nvfp4_stream_t stream) {
  clear_error();
  if (m > 0 && (!x || !gs_x)) return fail(NVFP4_ERR_INVALID_ARG, "nvfp4_quantize_gemm: null pointer");
  if (m > 0 && ldx < k)
    return fail(NVFP4_ERR_INVALID_ARG, "nvfp4_quantize_gemm: ldx=%lld < k=%lld", (long long)ldx, (long long)k);
  if (m > 0 && (!aligned(x, 16) || ldx % 8 || !aligned(gs_x, 4)))
    return fail(NVFP4_ERR_MISALIGNED, "nvfp4_quantize_gemm: x needs 16-B alignment and ldx %% 8 == 0");
  return run_gemm("nvfp4_quantize_gemm", nullptr, nullptr, b, sfb, alpha, d, m, n, k, workspace, workspace_bytes,
                  flags, stream, FusedA{static_cast<const __nv_bfloat16 *>(x), ldx, gs_x});
}
