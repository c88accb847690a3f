// The gated product of a feed-forward block, h = act(a0 A Bg^T) * (a1 A Bu^T), and its backward pass:
// the dense NVFP4 GEMM kernel (gemm.cuh) with another epilogue.
//
// The weight's rows alternate between 16 gate and 16 up rows, so that both products of an element of
// h meet in one tile: 32 neighbouring columns held by one thread where tokens fill the MMA's rows (and, turned
// around through shared memory, where the weight does and K is not split), units u and u + 4 of a split-K
// partial otherwise.
// The activation and the product are then taken on the fp32 accumulators and h is rounded once;
// neither product ever reaches memory.  The plans, pipelines and split reductions are the plain
// GEMM's.  The backward pass computes both products again from the packed operands (reading
// them costs 9/16 byte an element; storing both products for it would cost 4 bytes an element of h
// written and read) and turns dh into their gradients in the same epilogue.
#include "dense.cuh"

using namespace nvfp4;

namespace {

// a and b of gate_act's q = g (a + b g^2): sqrt(8 / pi) and 0.044715 times it for GELU's tanh form
bool activation_of(int activation, Gated &g) {
  if (activation == NVFP4_ACT_SILU) {
    g.act_a = 1.0f;
    g.act_b = 0.0f;
    return true;
  }
  if (activation == NVFP4_ACT_GELU_TANH) {
    g.act_a = 1.5957691216057308f;
    g.act_b = 0.044715f * 1.5957691216057308f;
    return true;
  }
  return false;
}

nvfp4_status_t check_gated(const char *name, int64_t inter, int activation, Gated &g) {
  if (inter <= 0 || inter >= (1LL << 30)) return fail(NVFP4_ERR_INVALID_ARG, "%s: inter=%lld", name, (long long)inter);
  if (inter % 16) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: inter=%lld is not a multiple of 16", name, (long long)inter);
  if (!activation_of(activation, g)) return fail(NVFP4_ERR_INVALID_ARG, "%s: activation=%d", name, activation);
  return NVFP4_OK;
}

}  // namespace

extern "C" nvfp4_status_t nvfp4_gated_gemm(const uint8_t *a, const uint8_t *sfa, const uint8_t *b, const uint8_t *sfb,
                                           const float *alpha, int activation, void *h, int64_t m, int64_t inter,
                                           int64_t k, void *workspace, size_t workspace_bytes, uint32_t flags,
                                           nvfp4_stream_t stream) {
  clear_error();
  Gated g{};
  const nvfp4_status_t st = check_gated("nvfp4_gated_gemm", inter, activation, g);
  if (st != NVFP4_OK) return st;
  return run_gemm<kEpiGated>("nvfp4_gated_gemm", a, sfa, b, sfb, alpha, h, m, 2 * inter, k, workspace, workspace_bytes, flags,
                             stream, FusedA{nullptr, 0, nullptr}, g);
}

extern "C" nvfp4_status_t nvfp4_gated_gemm_backward(const uint8_t *a, const uint8_t *sfa, const uint8_t *b,
                                                    const uint8_t *sfb, const float *alpha, int activation,
                                                    const void *dh, void *dgu, void *h, int64_t m, int64_t inter,
                                                    int64_t k, void *workspace, size_t workspace_bytes, uint32_t flags,
                                                    nvfp4_stream_t stream) {
  clear_error();
  const char *name = "nvfp4_gated_gemm_backward";
  Gated g{};
  const nvfp4_status_t st = check_gated(name, inter, activation, g);
  if (st != NVFP4_OK) return st;
  if (m > 0 && !dh) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!aligned(dh, 32) || !aligned(h, 32)) return fail(NVFP4_ERR_MISALIGNED, "%s: dh and h need 32-B alignment", name);
  g.dh = dh;
  g.h = h;
  return run_gemm<kEpiGatedGrad>(name, a, sfa, b, sfb, alpha, dgu, m, 2 * inter, k, workspace, workspace_bytes, flags, stream,
                                 FusedA{nullptr, 0, nullptr}, g);
}
