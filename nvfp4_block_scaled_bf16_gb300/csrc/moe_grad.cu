// Gradients of the MoE steps that move rows: of moe_combine (the experts' rows brought back with their weights) and
// of moe_gather_rows (the tokens' rows copied to the experts).  Both are bound by memory: one pass over the rows.
#include <cuda_bf16.h>

#include "host.h"
#include "ptx.cuh"

namespace nvfp4 {
namespace {

__device__ __forceinline__ void bf16x8(const uint4 &v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

constexpr int kSlots = 8;  // rows of a token that a thread has in flight
// Threads of a token's CTA: 256 took 53.8 us at 4096 tokens of 8 rows x 2048 channels, 128 take 44.6 (6.4 TB/s).
constexpr int kGradThreads = 128;

// With out[t] = sum_j w[t, j] y[pos[t, j]]:  dy[pos[t, j]] = w[t, j] dout[t],  dw[t, j] = dout[t] . y[pos[t, j]].
// One CTA a token, a thread 8 channels of every row: dout is read once (again from L1 past the first 8 slots), the
// rows of 8 slots are loaded together.  The dot products are summed in fp32: over a thread's channels in order,
// over the warp by exchanging halves (each step adds pairs of lanes and keeps half of the slots), over the warps in
// order, so the result does not depend on scheduling.
__global__ void __launch_bounds__(kGradThreads) moe_combine_grad_kernel(const uint4 *__restrict__ dout, int64_t ldo16,
                                                               const uint4 *__restrict__ y, int64_t rows,
                                                               const int32_t *__restrict__ pos, const float *__restrict__ w,
                                                               int topk, int pieces, uint4 *__restrict__ dy,
                                                               float *__restrict__ dw, unsigned int *status) {
  __shared__ float s_dot[kGradThreads / 32][kSlots];
  pdl_trigger();
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
  for (int j0 = 0; j0 < topk; j0 += kSlots) {
    int64_t p[kSlots];
    float wj[kSlots], dot[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      p[j] = -1;
      wj[j] = dot[j] = 0.0f;
      if (j0 + j < topk) {
        p[j] = pos[t * topk + j0 + j];
        wj[j] = w[t * topk + j0 + j];
        if (p[j] >= rows) {
          if (threadIdx.x == 0) atomicOr(status, 8u);
          p[j] = -1;
        }
      }
    }
    for (int c = threadIdx.x; c < pieces; c += blockDim.x) {
      uint4 v[kSlots];
      const uint4 o = __ldg(dout + t * ldo16 + c);
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (p[j] >= 0) v[j] = __ldg(y + p[j] * pieces + c);
      float g[8];
      bf16x8(o, g);
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        if (p[j] < 0) continue;
        float f[8];
        bf16x8(v[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[j] = fmaf(g[i], f[i], dot[j]);
        uint4 r;
        uint32_t *rp = &r.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) rp[i] = pack_bf16x2(wj[j] * g[2 * i], wj[j] * g[2 * i + 1]);
        dy[p[j] * pieces + c] = r;
      }
    }
    // eight sums over 32 lanes: 4 + 2 + 1 exchanges leave one slot's sum over 8 lanes in each lane, two more end it
#pragma unroll
    for (int half = kSlots / 2, o = 16; half >= 1; half >>= 1, o >>= 1) {
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int j = 0; j < half; ++j) {
        const float send = up ? dot[j] : dot[j + half];
        const float keep = up ? dot[j + half] : dot[j];
        dot[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
      }
    }
    dot[0] += __shfl_xor_sync(0xFFFFFFFFu, dot[0], 2);
    dot[0] += __shfl_xor_sync(0xFFFFFFFFu, dot[0], 1);
    if ((lane & 3) == 0) s_dot[warp][lane >> 2] = dot[0];  // lane bits 4, 3, 2 are the slot's bits 2, 1, 0
    __syncthreads();
    if (threadIdx.x < kSlots && j0 + static_cast<int>(threadIdx.x) < topk) {
      float s = s_dot[0][threadIdx.x];
      for (int i = 1; i < warps; ++i) s += s_dot[i][threadIdx.x];
      dw[t * topk + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

// With xs[r] = x[src[r]]:  dx[t] = sum_j dxs[pos[t, j]], fp32 sums in slot order, one rounding.  A thread sums 8
// channels of a token, the rows of 8 slots loaded together.  4096 tokens of 8 rows x 2048 channels: 25.4 us (5.9 TB/s).
template <typename I>
__global__ void __launch_bounds__(256) moe_gather_grad_kernel(const uint4 *__restrict__ dxs, int64_t rows,
                                                              const int32_t *__restrict__ pos, int64_t T, int topk,
                                                              int64_t pieces_, uint4 *__restrict__ dx, unsigned int *status) {
  pdl_trigger();
  pdl_wait();
  const I pieces = static_cast<I>(pieces_), total = static_cast<I>(T * pieces_);
  const I stride = static_cast<I>(gridDim.x) * blockDim.x;
  for (I i = static_cast<I>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += stride) {
    const I t_ = i / pieces;
    const int64_t t = t_, c = i - t_ * pieces;
    float acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = 0.0f;
    for (int j0 = 0; j0 < topk; j0 += kSlots) {
      uint4 v[kSlots];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        v[j] = make_uint4(0u, 0u, 0u, 0u);
        if (j0 + j < topk) {
          const int64_t p = pos[t * topk + j0 + j];
          if (p >= rows) {
            if (c == 0) atomicOr(status, 8u);
          } else if (p >= 0) {
            v[j] = __ldg(dxs + p * pieces_ + c);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        float f[8];
        bf16x8(v[j], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] += f[q];
      }
    }
    uint4 o;
    uint32_t *op = &o.x;
#pragma unroll
    for (int q = 0; q < 4; ++q) op[q] = pack_bf16x2(acc[2 * q], acc[2 * q + 1]);
    dx[t * pieces_ + c] = o;
  }
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status_t moe_combine_backward(const void *dout, int64_t ldo, const void *y, int64_t rows, const int32_t *pos,
                                               const float *weights, int64_t num_tokens, int topk, int64_t h, void *dy,
                                               float *dweights, uint32_t flags, nvfp4_stream_t stream) {
  clear_error();
  if (num_tokens < 0 || num_tokens >= (1LL << 31) || rows < 0 || topk < 1 || h <= 0 || h % 8 || h >= (1LL << 31) ||
      (ldo != 0 && ldo < h) || ldo % 8)
    return fail(NVFP4_ERR_INVALID_ARG, "moe_combine_backward: tokens=%lld rows=%lld topk=%d h=%lld ldo=%lld (h, ldo multiples of 8)",
                (long long)num_tokens, (long long)rows, topk, (long long)h, (long long)ldo);
  if (flags & ~(uint32_t)NVFP4_FLAG_PDL) return fail(NVFP4_ERR_INVALID_ARG, "moe_combine_backward: unknown flags 0x%x", flags);
  if (num_tokens == 0) return NVFP4_OK;
  if (!dout || !pos || !weights || !dweights || (rows > 0 && (!y || !dy)))
    return fail(NVFP4_ERR_INVALID_ARG, "moe_combine_backward: null pointer");
  if (rows > 0 && y == dy) return fail(NVFP4_ERR_INVALID_ARG, "moe_combine_backward: dy must not be y");
  if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16) || !aligned(pos, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
    return fail(NVFP4_ERR_MISALIGNED, "moe_combine_backward: dout, y and dy need 16-B, pos and the weights 4-B alignment");
  DeviceInfo dev;
  nvfp4_status_t st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  const int pieces = static_cast<int>(h / 8);
  const int threads = pieces >= kGradThreads ? kGradThreads : static_cast<int>(round_up(pieces, 32));
  cudaError_t e = launch(moe_combine_grad_kernel, dim3(static_cast<unsigned>(num_tokens)), dim3(threads), 0, (cudaStream_t)stream,
                         (flags & NVFP4_FLAG_PDL) != 0, 1, static_cast<const uint4 *>(dout), ldo / 8, static_cast<const uint4 *>(y),
                         rows, pos, weights, topk, pieces, static_cast<uint4 *>(dy), dweights, dev.status);
  return check_launch(e, "moe_combine_backward");
}

extern "C" nvfp4_status_t moe_gather_backward(const void *dxs, int64_t rows, const int32_t *pos, int64_t num_tokens, int topk,
                                              int64_t h, void *dx, uint32_t flags, nvfp4_stream_t stream) {
  clear_error();
  if (num_tokens < 0 || num_tokens >= (1LL << 31) || rows < 0 || topk < 1 || h <= 0 || h % 8 || h >= (1LL << 31))
    return fail(NVFP4_ERR_INVALID_ARG, "moe_gather_backward: tokens=%lld rows=%lld topk=%d h=%lld (h a multiple of 8)",
                (long long)num_tokens, (long long)rows, topk, (long long)h);
  if (flags & ~(uint32_t)NVFP4_FLAG_PDL) return fail(NVFP4_ERR_INVALID_ARG, "moe_gather_backward: unknown flags 0x%x", flags);
  if (num_tokens == 0) return NVFP4_OK;
  if (!pos || !dx || (rows > 0 && !dxs)) return fail(NVFP4_ERR_INVALID_ARG, "moe_gather_backward: null pointer");
  if (!aligned(dxs, 16) || !aligned(dx, 16) || !aligned(pos, 4))
    return fail(NVFP4_ERR_MISALIGNED, "moe_gather_backward: dxs and dx need 16-B, pos 4-B alignment");
  DeviceInfo dev;
  nvfp4_status_t st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  const int64_t pieces = h / 8, blocks = ceil_div(num_tokens * pieces, 256), cap = dev.sm_count * 8LL;
  const int grid = static_cast<int>(blocks < cap ? blocks : cap);
  auto kern = fits_i32_loop(num_tokens * pieces, grid * 256LL) ? moe_gather_grad_kernel<int> : moe_gather_grad_kernel<int64_t>;
  cudaError_t e = launch(kern, dim3(grid), dim3(256), 0, (cudaStream_t)stream, (flags & NVFP4_FLAG_PDL) != 0, 1,
                         static_cast<const uint4 *>(dxs), rows, pos, num_tokens, topk, pieces, static_cast<uint4 *>(dx), dev.status);
  return check_launch(e, "moe_gather_backward");
}
