// RMS norms around a decoder block, fused with the block's gate and residual sum (forward, forward
// with NVFP4 output, backward).
//
// Forward, one row of n channels:
//   p = y * rsqrt(mean(y^2) + eps) * (offset + w_post)      the norm after the block (p = y without w_post)
//   r = x + scale * (gate * p)                              the residual stream, stored in x's type
//   h = r * rsqrt(mean(r^2) + eps) * (offset + w_pre)       the norm before the next block
// in fp32; r is rounded once, when it is stored, and h is computed from the unrounded r.  The
// NVFP4 form quantises bf16(h) with the arithmetic of nvfp4_quantize, so it equals the two calls.
//
// Backward, from the stored stream r and the block's output y; dr is the gradient that reaches r
// from the rest of the network, dh the one that reaches h, xn = r * rstd_r, yn = y * rstd_y:
//   d    = dh * (offset + w_pre)
//   g    = dr + rstd_r * (d - xn * mean(d * xn))            gradient of x (and of r)
//   dw_pre  = sum over rows of dh * xn
//   dgate   = scale * g * yn * (offset + w_post)            (summed over rows for a channel gate)
//   b    = scale * g * gate;  dw_post = sum over rows of b * yn
//   e    = b * (offset + w_post);  dy = rstd_y * (e - yn * mean(e * yn))
//
// Every kernel reads each input once and keeps the row in registers between the two reductions:
// they are bound by memory for many rows and by latency for few.  A team (a warp up to 512
// channels, otherwise a block) owns a row; a thread holds 8 * VPT of its channels.
#include <cuda_bf16.h>

#include "host.h"
#include "ptx.cuh"

namespace nvfp4 {
namespace {

constexpr int kMaxChannels = 32768;  // 1024 threads x 8 channels x 4
constexpr int kWarpTeams = 8;        // rows per block where a warp owns a row

struct NormArgs {
  const void *x;
  int64_t ldx;
  const __nv_bfloat16 *y;
  int64_t ldy;
  const __nv_bfloat16 *w_post, *w_pre;
  const __nv_bfloat16 *gate;
  int64_t ldg;  // 0: one gate per channel, shared by every row
  float scale, eps, offset;
  void *x_out;
  int64_t ldxo;
  __nv_bfloat16 *h;
  int64_t ldh;
  const float *gs;
  uint8_t *q, *sf;
  int64_t m;
  int n;
  int cp;  // NVFP4 output: scale columns, round_up(n / 16, 4)
};

// Channels of a row that one thread of a team holds.  VEC (every row 16-byte aligned, n a multiple
// of 8): 8 adjacent channels per step, so that a thread loads and stores 16 bytes of bf16; otherwise
// single channels, neighbours in neighbouring threads.
template <bool VEC>
__device__ __forceinline__ int channel(int i, int t, int ts) {
  return VEC ? ((i >> 3) * ts + t) * 8 + (i & 7) : i * ts + t;
}

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *f) {
  const uint4 v = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float *p, float *f) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *f) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                             pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store8(float *p, const float *f) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }

// Channels past n read as zero, and so add nothing to any sum below.
template <int VPT, bool VEC, typename T>
__device__ __forceinline__ void load_row(const T *row, float (&f)[8 * VPT], int t, int ts, int n) {
  if constexpr (VEC) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * ts + t) * 8;
      if (c < n) {
        load8(row + c, f + 8 * v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[8 * v + i] = 0.0f;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8 * VPT; ++i) {
      const int c = i * ts + t;
      f[i] = c < n ? to_f32(row[c]) : 0.0f;
    }
  }
}
template <int VPT, bool VEC, typename T>
__device__ __forceinline__ void store_row(T *row, const float (&f)[8 * VPT], int t, int ts, int n) {
  if constexpr (VEC) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * ts + t) * 8;
      if (c < n) store8(row + c, f + 8 * v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8 * VPT; ++i) {
      const int c = i * ts + t;
      if (c < n) put(row + c, f[i]);
    }
  }
}

// Sums of N values over a team, in an order fixed by the team's size.  A block passes them through
// one of two shared buffers: two sums in a row use different ones, so one barrier each is enough (a
// buffer is written again only after the barrier of the sum in between, which every reader of the
// buffer has reached).
template <int N>
struct TeamSum {
  float (*buf)[N][32];  // [2][N][32], block teams only
  int which = 0;
  template <bool WARP>
  __device__ __forceinline__ void sum(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
    if constexpr (!WARP) {
      const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
      if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buf[which][i][warp] = v[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float s = lane < warps ? buf[which][i][lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        v[i] = s;
      }
      which ^= 1;
    }
  }
};

// NVFP4 of a row already rounded to bf16: a 16-channel block is the 8 channels of two neighbouring
// threads, and eight threads gather the four scale bytes of a 32-bit word of the 128x4 layout.
// Every lane of the warp takes part; channels past n (whole blocks) get zero scales.
template <int VPT>
__device__ __forceinline__ void quantize_row(const NormArgs &p, const float (&f)[8 * VPT], int64_t row, int t, int ts) {
  const float gs = __ldg(p.gs);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (v * ts + t) * 8;
    float amax = 0.0f, y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[8 * v + i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    uint32_t code = 0;
    const float inv = nvfp4_block_scale(amax, gs, code);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(f[8 * v + i], inv);
    if (c < p.n) *reinterpret_cast<uint32_t *>(p.q + row * (p.n >> 1) + (c >> 1)) = e2m1x8(y);
    else code = 0;
    const uint32_t b1 = __shfl_down_sync(0xFFFFFFFFu, code, 2);
    const uint32_t b2 = __shfl_down_sync(0xFFFFFFFFu, code, 4);
    const uint32_t b3 = __shfl_down_sync(0xFFFFFFFFu, code, 6);
    const int j = c >> 4;  // scale column
    if ((t & 7) == 0 && j < p.cp)
      *reinterpret_cast<uint32_t *>(p.sf + ((row >> 7) * (p.cp >> 2) + (j >> 2)) * 512 + (row & 31) * 16 +
                                    ((row >> 5) & 3) * 4) = code | (b1 << 8) | (b2 << 16) | (b3 << 24);
  }
}

// Blocks [0, row_blocks) hold the rows; with NVFP4 output the blocks after them zero the scale rows
// between m and the next multiple of 128.
// MAXT: threads of the largest block it is launched with (512 or 1024: 128 or 64 registers).
template <typename XT, int VPT, bool VEC, bool WARP, bool QUANT, int MAXT>
__global__ void __launch_bounds__(WARP ? 32 * kWarpTeams : MAXT)
    norm_kernel(const NormArgs p, unsigned int row_blocks) {
  __shared__ float s_buf[2][1][32];
  // The next kernel may launch now: it waits for this grid before it reads what is written here.
  pdl_trigger();
  pdl_wait();
  if (QUANT && blockIdx.x >= row_blocks) {
    const int64_t words = ((p.m + 127) / 128 * 128 - p.m) * (p.cp >> 2);
    const int64_t stride = static_cast<int64_t>(gridDim.x - row_blocks) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x - row_blocks) * blockDim.x + threadIdx.x; i < words; i += stride) {
      const int64_t row = p.m + i / (p.cp >> 2), jt = i % (p.cp >> 2);
      *reinterpret_cast<uint32_t *>(p.sf + ((row >> 7) * (p.cp >> 2) + jt) * 512 + (row & 31) * 16 +
                                    ((row >> 5) & 3) * 4) = 0u;
    }
    return;
  }
  const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpTeams + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= p.m) return;
  const int t = WARP ? threadIdx.x & 31 : threadIdx.x, ts = WARP ? 32 : blockDim.x;
  constexpr int E = 8 * VPT;
  TeamSum<1> team{s_buf};
  const float inv_n = 1.0f / static_cast<float>(p.n);
  float r[E], w[E];
  load_row<VPT, VEC>(static_cast<const XT *>(p.x) + row * p.ldx, r, t, ts, p.n);
  if (p.y) {
    float y[E];
    load_row<VPT, VEC>(p.y + row * p.ldy, y, t, ts, p.n);
    if (p.w_pre) load_row<VPT, VEC>(p.w_pre, w, t, ts, p.n);
    if (p.w_post) {
      float wp[E];
      load_row<VPT, VEC>(p.w_post, wp, t, ts, p.n);
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < E; ++i) s[0] += y[i] * y[i];
      team.template sum<WARP>(s);
      const float rstd = rsqrtf(s[0] * inv_n + p.eps);
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] = y[i] * rstd * (p.offset + wp[i]);
    }
    if (p.gate) {
      float g[E];
      load_row<VPT, VEC>(p.gate + row * p.ldg, g, t, ts, p.n);
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] *= g[i];
    }
#pragma unroll
    for (int i = 0; i < E; ++i) r[i] = r[i] + p.scale * y[i];
    store_row<VPT, VEC>(static_cast<XT *>(p.x_out) + row * p.ldxo, r, t, ts, p.n);
  } else {
    load_row<VPT, VEC>(p.w_pre, w, t, ts, p.n);
  }
  if (!p.w_pre) return;
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < E; ++i) s[0] += r[i] * r[i];
  team.template sum<WARP>(s);
  const float rstd = rsqrtf(s[0] * inv_n + p.eps);
#pragma unroll
  for (int i = 0; i < E; ++i) r[i] = r[i] * rstd * (p.offset + w[i]);
  if constexpr (QUANT) {
#pragma unroll
    for (int i = 0; i < E; ++i) r[i] = __bfloat162float(__float2bfloat16_rn(r[i]));
    quantize_row<VPT>(p, r, row, t, ts);
  } else {
    store_row<VPT, VEC>(p.h + row * p.ldh, r, t, ts, p.n);
  }
}

// ------------------------------------------------------------------ backward
struct NormGradArgs {
  const __nv_bfloat16 *dh;
  int64_t lddh;
  const void *dr;  // gradient of the stored stream, or nullptr for zero
  int64_t lddr;
  const void *r;   // the stored stream
  int64_t ldr;
  const __nv_bfloat16 *y;
  int64_t ldy;
  const __nv_bfloat16 *w_post, *w_pre, *gate;
  int64_t ldg;
  float scale, eps, offset;
  void *dx;
  int64_t lddx;
  __nv_bfloat16 *dy;
  int64_t lddy;
  __nv_bfloat16 *dgate;  // gate per token: [m, n]
  int64_t lddg;
  float *part;           // [teams][planes][n]: every team's sums over its rows
  int64_t m;
  int n, planes;         // planes: dw_pre, dw_post, dgate (those that are summed over rows), in this order
  int teams;
};

// Team k takes rows k, k + teams, ...; its column sums stay in registers and are written to its own
// row of the workspace, which norm_colsum_kernel adds up in order: no atomics, so the result does
// not depend on timing.
template <typename XT, int VPT, bool VEC, bool WARP, int MAXT>
__global__ void __launch_bounds__(WARP ? 32 * kWarpTeams : MAXT)
    norm_grad_kernel(const NormGradArgs p) {
  __shared__ float s_buf3[2][3][32];
  __shared__ float s_buf1[2][1][32];
  pdl_trigger();
  pdl_wait();
  const int teamid = WARP ? blockIdx.x * kWarpTeams + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && teamid >= p.teams) return;
  const int t = WARP ? threadIdx.x & 31 : threadIdx.x, ts = WARP ? 32 : blockDim.x;
  constexpr int E = 8 * VPT;
  TeamSum<3> team3{s_buf3};
  TeamSum<1> team1{s_buf1};
  const float inv_n = 1.0f / static_cast<float>(p.n);
  float aw[E], ap[E], ag[E];
#pragma unroll
  for (int i = 0; i < E; ++i) aw[i] = ap[i] = ag[i] = 0.0f;
  for (int64_t row = teamid; row < p.m; row += p.teams) {
    float r[E], d[E], g[E], y[E];
    load_row<VPT, VEC>(static_cast<const XT *>(p.r) + row * p.ldr, r, t, ts, p.n);
    if (p.dh) {
      load_row<VPT, VEC>(p.dh + row * p.lddh, d, t, ts, p.n);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) d[i] = 0.0f;
    }
    if (p.dr) {
      load_row<VPT, VEC>(static_cast<const XT *>(p.dr) + row * p.lddr, g, t, ts, p.n);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) g[i] = 0.0f;
    }
    if (p.y) {
      load_row<VPT, VEC>(p.y + row * p.ldy, y, t, ts, p.n);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] = 0.0f;
    }
    // sums of r^2, of (dh w) r and of y^2 in one go: mean(d xn) = rstd * sum(d r) / n
    float s[3] = {0.0f, 0.0f, 0.0f};
    {
      float w[E];
      if (p.dh) {
        load_row<VPT, VEC>(p.w_pre, w, t, ts, p.n);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) w[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        s[0] += r[i] * r[i];
        s[1] += d[i] * (p.offset + w[i]) * r[i];
        s[2] += y[i] * y[i];
      }
      team3.template sum<WARP>(s);
      const float rstd = rsqrtf(s[0] * inv_n + p.eps);
      const float mean = s[1] * rstd * inv_n;
      if (p.dh) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float xn = r[i] * rstd;
          aw[i] += d[i] * xn;
          g[i] += rstd * (d[i] * (p.offset + w[i]) - xn * mean);
        }
      }
    }
    store_row<VPT, VEC>(static_cast<XT *>(p.dx) + row * p.lddx, g, t, ts, p.n);
    if (!p.y) continue;
    const float rstd = p.w_post ? rsqrtf(s[2] * inv_n + p.eps) : 1.0f;
    float wp[E];
    if (p.w_post) {
      load_row<VPT, VEC>(p.w_post, wp, t, ts, p.n);
#pragma unroll
      for (int i = 0; i < E; ++i) wp[i] += p.offset;
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) wp[i] = 1.0f;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      g[i] *= p.scale;
      y[i] *= rstd;
    }
    if (p.gate) {
      load_row<VPT, VEC>(p.gate + row * p.ldg, d, t, ts, p.n);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        r[i] = g[i] * y[i] * wp[i];
        g[i] *= d[i];
      }
      if (p.ldg != 0) {
        store_row<VPT, VEC>(p.dgate + row * p.lddg, r, t, ts, p.n);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) ag[i] += r[i];
      }
    }
    if (p.w_post) {
      float q[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < E; ++i) {
        ap[i] += g[i] * y[i];
        g[i] *= wp[i];
        q[0] += g[i] * y[i];
      }
      team1.template sum<WARP>(q);
      const float mean = q[0] * inv_n;
#pragma unroll
      for (int i = 0; i < E; ++i) g[i] = rstd * (g[i] - y[i] * mean);
    }
    store_row<VPT, VEC>(p.dy + row * p.lddy, g, t, ts, p.n);
  }
  float *part = p.part + static_cast<int64_t>(teamid) * p.planes * p.n;
  if (p.dh) {
    store_row<VPT, VEC>(part, aw, t, ts, p.n);
    part += p.n;
  }
  if (p.y && p.w_post) {
    store_row<VPT, VEC>(part, ap, t, ts, p.n);
    part += p.n;
  }
  if (p.y && p.gate && p.ldg == 0) store_row<VPT, VEC>(part, ag, t, ts, p.n);
}

// out[plane][c] = sum over teams of part[team][plane][c]: 32 columns a block, each of its 32 warps
// sums every 32nd team, then the warps' sums are added in warp order.
__global__ void __launch_bounds__(1024) norm_colsum_kernel(const float *__restrict__ part, int teams, int planes, int n,
                                                           float *o0, float *o1, float *o2) {
  __shared__ float s[32][33];
  pdl_trigger();
  pdl_wait();
  const int64_t cols = static_cast<int64_t>(planes) * n;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float v = 0.0f;
  if (col < cols) {
    int k = threadIdx.y;
    for (; k + 96 < teams; k += 128) {  // four loads in flight
      const float a = part[k * cols + col], b = part[(k + 32) * cols + col];
      const float c = part[(k + 64) * cols + col], d = part[(k + 96) * cols + col];
      v += (a + b) + (c + d);
    }
    for (; k < teams; k += 32) v += part[k * cols + col];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0 || col >= cols) return;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) sum += s[i][threadIdx.x];
  const int plane = static_cast<int>(col / n);
  (plane == 0 ? o0 : plane == 1 ? o1 : o2)[col - static_cast<int64_t>(plane) * n] = sum;
}

// How a row is spread over threads.
struct Shape {
  bool warp;
  int vpt, threads;
};
// n channels as vectors of 8 (n_pad >= n: channels the NVFP4 scale columns need).  A warp owns a
// row up to 512 channels; a block otherwise, with `vpt_pref` vectors a thread where 1024 threads allow.
Shape shape_of(int64_t n_pad, int vpt_pref) {
  const int nv = static_cast<int>(ceil_div(n_pad, 8));
  if (nv <= 32) return {true, 1, 32 * kWarpTeams};
  if (nv <= 64) return {true, 2, 32 * kWarpTeams};
  int vpt = vpt_pref;
  while (nv > 1024 * vpt) vpt *= 2;
  return {false, vpt, static_cast<int>(round_up(ceil_div(nv, vpt), 32))};
}

template <typename XT, bool VEC, bool QUANT, int MAXT>
auto forward_block(int vpt) {
  return vpt == 1 ? norm_kernel<XT, 1, VEC, false, QUANT, MAXT>
                  : (vpt == 2 ? norm_kernel<XT, 2, VEC, false, QUANT, MAXT> : norm_kernel<XT, 4, VEC, false, QUANT, MAXT>);
}
template <typename XT, bool VEC, bool QUANT>
auto forward_kernel(const Shape &s) {
  if (s.warp) return s.vpt == 1 ? norm_kernel<XT, 1, VEC, true, QUANT, 512> : norm_kernel<XT, 2, VEC, true, QUANT, 512>;
  return s.threads <= 512 ? forward_block<XT, VEC, QUANT, 512>(s.vpt) : forward_block<XT, VEC, QUANT, 1024>(s.vpt);
}
template <typename XT, bool VEC, int MAXT>
auto backward_block(int vpt) {
  return vpt == 1 ? norm_grad_kernel<XT, 1, VEC, false, MAXT>
                  : (vpt == 2 ? norm_grad_kernel<XT, 2, VEC, false, MAXT> : norm_grad_kernel<XT, 4, VEC, false, MAXT>);
}
template <typename XT, bool VEC>
auto backward_kernel(const Shape &s) {
  if (s.warp) return s.vpt == 1 ? norm_grad_kernel<XT, 1, VEC, true, 512> : norm_grad_kernel<XT, 2, VEC, true, 512>;
  return s.threads <= 512 ? backward_block<XT, VEC, 512>(s.vpt) : backward_block<XT, VEC, 1024>(s.vpt);
}

// Teams of the backward pass: enough to fill the SMs, each with a row of its own.  (Fixed per shape
// and device, so that the order of the column sums is too.)
int grad_teams(int64_t m, const Shape &s, int sm_count) {
  const int64_t per_sm = s.warp ? 4 * kWarpTeams : (s.threads <= 512 ? 2 : 1);
  const int64_t cap = per_sm * sm_count;
  return static_cast<int>(m < cap ? m : cap);
}

bool rows_aligned(const void *p, int64_t ld, int elem) { return !p || (aligned(p, 16) && ld * elem % 16 == 0); }
// Row stride of an input: 0 (one row for all) or at least a row.
bool in_stride(int64_t ld, int64_t n) { return ld == 0 || ld >= n; }
int elem_of(int type) { return type == NVFP4_DTYPE_F32 ? 4 : 2; }

// The checks that the forward entry points share.
nvfp4_status_t check_norm(const char *name, const void *x, int x_type, int64_t ldx, const void *y, int64_t ldy,
                          const void *w_post, const void *gate, int64_t ldg, const void *w_pre, const void *x_out,
                          int64_t ldxo, int64_t m, int64_t n, uint32_t flags) {
  if (m < 0 || n <= 0 || m >= (1LL << 31)) return fail(NVFP4_ERR_INVALID_ARG, "%s: m=%lld n=%lld", name, (long long)m, (long long)n);
  if (n > kMaxChannels) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: n=%lld (at most %d)", name, (long long)n, kMaxChannels);
  if (x_type != NVFP4_DTYPE_BF16 && x_type != NVFP4_DTYPE_F32) return fail(NVFP4_ERR_INVALID_ARG, "%s: x_type=%d", name, x_type);
  if (flags & ~(uint32_t)NVFP4_FLAG_PDL) return fail(NVFP4_ERR_INVALID_ARG, "%s: unknown flags 0x%x", name, flags);
  if (m == 0) return NVFP4_OK;  // (an empty operand may come without an address)
  if (!y && (w_post || gate || x_out))
    return fail(NVFP4_ERR_INVALID_ARG, "%s: w_post, gate and x_out belong to y, which is NULL", name);
  if (!y && !w_pre) return fail(NVFP4_ERR_INVALID_ARG, "%s: neither y nor w_pre: nothing to compute", name);
  if (!in_stride(ldx, n) || (y && !in_stride(ldy, n)) || (gate && !in_stride(ldg, n)) || (x_out && ldxo < n))
    return fail(NVFP4_ERR_INVALID_ARG, "%s: row strides ldx=%lld ldy=%lld ldg=%lld ldxo=%lld are shorter than n=%lld", name,
                (long long)ldx, (long long)ldy, (long long)ldg, (long long)ldxo, (long long)n);
  if (!x || (y && !x_out)) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", name);
  const int xe = elem_of(x_type);
  if (!aligned(x, xe) || !aligned(x_out, xe) || !aligned(y, 2) || !aligned(w_post, 2) || !aligned(gate, 2) || !aligned(w_pre, 2))
    return fail(NVFP4_ERR_MISALIGNED, "%s: a pointer is not aligned to its element", name);
  return NVFP4_OK;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

// One vector a thread while the rows are few (the call waits for one row's latency: 7168 channels,
// one row), two from four rows an SM on (fewer, wider threads: more bytes in flight per warp).
static int forward_vpt(int64_t m, int64_t n, int sm_count) { return m >= 4LL * sm_count && n > 2048 ? 2 : 1; }

extern "C" nvfp4_status_t block_norm(const void *x, int x_type, int64_t ldx, const void *y, int64_t ldy,
                                     const void *w_post, const void *gate, int64_t ldg, const void *w_pre,
                                     float residual_scale, float eps, float weight_offset, void *x_out, int64_t ldxo,
                                     void *h, int64_t ldh, int64_t m, int64_t n, uint32_t flags,
                                     nvfp4_stream_t stream) {
  clear_error();
  nvfp4_status_t st = check_norm("block_norm", x, x_type, ldx, y, ldy, w_post, gate, ldg, w_pre, x_out, ldxo, m, n, flags);
  if (st != NVFP4_OK) return st;
  if ((w_pre != nullptr) != (h != nullptr) && m > 0)
    return fail(NVFP4_ERR_INVALID_ARG, "block_norm: h is the norm with w_pre: give both or neither");
  if (h && ldh < n) return fail(NVFP4_ERR_INVALID_ARG, "block_norm: ldh=%lld < n=%lld", (long long)ldh, (long long)n);
  if (m == 0) return NVFP4_OK;
  if (!aligned(h, 2)) return fail(NVFP4_ERR_MISALIGNED, "block_norm: a pointer is not aligned to its element");
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  const int xe = elem_of(x_type);
  const bool vec = n % 8 == 0 && rows_aligned(x, ldx, xe) && rows_aligned(y, ldy, 2) && rows_aligned(gate, ldg, 2) &&
                   rows_aligned(x_out, ldxo, xe) && rows_aligned(h, ldh, 2) && aligned(w_post, 16) && aligned(w_pre, 16);
  const Shape s = shape_of(n, forward_vpt(m, n, dev.sm_count));
  NormArgs a{x, ldx, (const __nv_bfloat16 *)y, ldy, (const __nv_bfloat16 *)w_post, (const __nv_bfloat16 *)w_pre,
             (const __nv_bfloat16 *)gate, ldg, residual_scale, eps, weight_offset, x_out, ldxo, (__nv_bfloat16 *)h, ldh,
             nullptr, nullptr, nullptr, m, static_cast<int>(n), 0};
  const bool f32 = x_type == NVFP4_DTYPE_F32;
  auto kern = f32 ? (vec ? forward_kernel<float, true, false>(s) : forward_kernel<float, false, false>(s))
                  : (vec ? forward_kernel<__nv_bfloat16, true, false>(s) : forward_kernel<__nv_bfloat16, false, false>(s));
  const unsigned int rows = static_cast<unsigned int>(s.warp ? ceil_div(m, kWarpTeams) : m);
  return check_launch(launch(kern, dim3(rows), dim3(s.threads), 0, (cudaStream_t)stream, (flags & NVFP4_FLAG_PDL) != 0, 1,
                             a, rows), "block_norm");
}

extern "C" nvfp4_status_t block_norm_quantize(const void *x, int x_type, int64_t ldx, const void *y, int64_t ldy,
                                              const void *w_post, const void *gate, int64_t ldg, const void *w_pre,
                                              float residual_scale, float eps, float weight_offset, void *x_out,
                                              int64_t ldxo, const float *gs, uint8_t *q, uint8_t *sf, int64_t m,
                                              int64_t n, uint32_t flags, nvfp4_stream_t stream) {
  clear_error();
  const char *name = "block_norm_quantize";
  nvfp4_status_t st = check_norm(name, x, x_type, ldx, y, ldy, w_post, gate, ldg, w_pre, x_out, ldxo, m, n, flags);
  if (st != NVFP4_OK) return st;
  if (n % 16) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: n=%lld is not a multiple of 16", name, (long long)n);
  if (m == 0) return NVFP4_OK;
  if (!w_pre || !gs || !q || !sf) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", name);
  const int xe = elem_of(x_type);
  if (!rows_aligned(x, ldx, xe) || !rows_aligned(y, ldy, 2) || !rows_aligned(gate, ldg, 2) ||
      !rows_aligned(x_out, ldxo, xe) || !aligned(w_post, 16) || !aligned(w_pre, 16) || !aligned(sf, 16) || !aligned(q, 8) ||
      !aligned(gs, 4))
    return fail(NVFP4_ERR_MISALIGNED, "%s: every row of x, y, gate, x_out, the weights and sf need 16-B, q 8-B, gs 4-B alignment", name);
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  const int64_t cp = round_up(n / 16, 4);
  const Shape s = shape_of(cp * 16, forward_vpt(m, n, dev.sm_count));
  NormArgs a{x, ldx, (const __nv_bfloat16 *)y, ldy, (const __nv_bfloat16 *)w_post, (const __nv_bfloat16 *)w_pre,
             (const __nv_bfloat16 *)gate, ldg, residual_scale, eps, weight_offset, x_out, ldxo, nullptr, 0,
             gs, q, sf, m, static_cast<int>(n), static_cast<int>(cp)};
  auto kern = x_type == NVFP4_DTYPE_F32 ? forward_kernel<float, true, true>(s) : forward_kernel<__nv_bfloat16, true, true>(s);
  const unsigned int rows = static_cast<unsigned int>(s.warp ? ceil_div(m, kWarpTeams) : m);
  const int64_t words = (round_up(m, 128) - m) * (cp / 4);
  const int64_t pad = ceil_div(words, s.threads);
  const unsigned int extra = static_cast<unsigned int>(pad < dev.sm_count ? pad : dev.sm_count);
  return check_launch(launch(kern, dim3(rows + extra), dim3(s.threads), 0, (cudaStream_t)stream,
                             (flags & NVFP4_FLAG_PDL) != 0, 1, a, rows), name);
}

extern "C" size_t block_norm_backward_workspace_size(int64_t m, int64_t n) {
  if (m < 0 || n <= 0 || n > kMaxChannels) return 0;
  // (the largest number of teams on any GPU this library runs on; sized without a device)
  return static_cast<size_t>(grad_teams(m, shape_of(n, 1), 160)) * 3 * static_cast<size_t>(n) * 4;
}

extern "C" nvfp4_status_t block_norm_backward(const void *dh, int64_t lddh, const void *dx_out, int64_t lddxo,
                                              const void *x_out, int x_type, int64_t ldxo, const void *y, int64_t ldy,
                                              const void *w_post, const void *gate, int64_t ldg, const void *w_pre,
                                              float residual_scale, float eps, float weight_offset, void *dx,
                                              int64_t lddx, void *dy, int64_t lddy, float *dw_pre, float *dw_post,
                                              void *dgate, int64_t lddg, int64_t m, int64_t n, void *workspace,
                                              size_t workspace_bytes, uint32_t flags, nvfp4_stream_t stream) {
  clear_error();
  const char *name = "block_norm_backward";
  if (m < 0 || n <= 0 || m >= (1LL << 31)) return fail(NVFP4_ERR_INVALID_ARG, "%s: m=%lld n=%lld", name, (long long)m, (long long)n);
  if (n > kMaxChannels) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: n=%lld (at most %d)", name, (long long)n, kMaxChannels);
  if (x_type != NVFP4_DTYPE_BF16 && x_type != NVFP4_DTYPE_F32) return fail(NVFP4_ERR_INVALID_ARG, "%s: x_type=%d", name, x_type);
  if (flags & ~(uint32_t)NVFP4_FLAG_PDL) return fail(NVFP4_ERR_INVALID_ARG, "%s: unknown flags 0x%x", name, flags);
  if (m > 0 && !y && (w_post || gate || dy || dw_post || dgate))  // (an empty y may come without an address)
    return fail(NVFP4_ERR_INVALID_ARG, "%s: w_post, gate, dy, dw_post and dgate belong to y, which is NULL", name);
  if ((dh != nullptr) != (w_pre != nullptr) && m > 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: dh and w_pre: give both or neither", name);
  const bool token_gate = gate && ldg != 0;
  if (!in_stride(ldxo, n) || lddx < n || (dh && !in_stride(lddh, n)) || (dx_out && !in_stride(lddxo, n)) ||
      (y && (!in_stride(ldy, n) || lddy < n)) || (token_gate && (ldg < n || lddg < n)))
    return fail(NVFP4_ERR_INVALID_ARG, "%s: a row stride is shorter than n=%lld", name, (long long)n);
  if ((w_pre != nullptr) != (dw_pre != nullptr) || (w_post != nullptr) != (dw_post != nullptr) ||
      (gate != nullptr) != (dgate != nullptr))
    return fail(NVFP4_ERR_INVALID_ARG, "%s: dw_pre, dw_post and dgate: one for each of w_pre, w_post and gate", name);
  if (m > 0 && (!x_out || !dx || (y && !dy))) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", name);
  const int xe = elem_of(x_type), ge = token_gate ? 2 : 4;
  if (!aligned(x_out, xe) || !aligned(dx, xe) || !aligned(dx_out, xe) || !aligned(dh, 2) || !aligned(y, 2) || !aligned(dy, 2) ||
      !aligned(w_post, 2) || !aligned(w_pre, 2) || !aligned(gate, 2) || !aligned(dw_pre, 4) || !aligned(dw_post, 4) ||
      !aligned(dgate, ge))
    return fail(NVFP4_ERR_MISALIGNED, "%s: a pointer is not aligned to its element", name);
  const bool channel_gate = gate && !token_gate;
  const int planes = (w_pre ? 1 : 0) + (w_post ? 1 : 0) + (channel_gate ? 1 : 0);
  const size_t need = planes ? block_norm_backward_workspace_size(m, n) : 0;
  if (need && (!workspace || workspace_bytes < need))
    return fail(NVFP4_ERR_INVALID_ARG, "%s: needs a workspace of %zu bytes (got %zu%s)", name, need, workspace_bytes,
                workspace ? "" : ", NULL");
  if (!aligned(workspace, 16)) return fail(NVFP4_ERR_MISALIGNED, "%s: workspace needs 16-B alignment", name);
  if (m == 0 && planes == 0) return NVFP4_OK;
  DeviceInfo dev;
  nvfp4_status_t st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  const bool vec = n % 8 == 0 && rows_aligned(dh, lddh, 2) && rows_aligned(dx_out, lddxo, xe) && rows_aligned(x_out, ldxo, xe) &&
                   rows_aligned(y, ldy, 2) && rows_aligned(gate, ldg, 2) && rows_aligned(dx, lddx, xe) &&
                   rows_aligned(dy, lddy, 2) && (!token_gate || rows_aligned(dgate, lddg, 2)) && aligned(w_post, 16) &&
                   aligned(w_pre, 16);
  const Shape s = shape_of(n, 1);
  const int teams = grad_teams(m, s, dev.sm_count < 160 ? dev.sm_count : 160);
  NormGradArgs a{(const __nv_bfloat16 *)dh, lddh, dx_out, lddxo, x_out, ldxo, (const __nv_bfloat16 *)y, ldy,
                 (const __nv_bfloat16 *)w_post, (const __nv_bfloat16 *)w_pre, (const __nv_bfloat16 *)gate, ldg,
                 residual_scale, eps, weight_offset, dx, lddx, (__nv_bfloat16 *)dy, lddy,
                 token_gate ? (__nv_bfloat16 *)dgate : nullptr, lddg, static_cast<float *>(workspace), m,
                 static_cast<int>(n), planes, teams};
  const bool pdl = (flags & NVFP4_FLAG_PDL) != 0, f32 = x_type == NVFP4_DTYPE_F32;
  cudaError_t e = cudaSuccess;
  if (m > 0) {
    auto kern = f32 ? (vec ? backward_kernel<float, true>(s) : backward_kernel<float, false>(s))
                    : (vec ? backward_kernel<__nv_bfloat16, true>(s) : backward_kernel<__nv_bfloat16, false>(s));
    e = launch(kern, dim3(static_cast<unsigned>(s.warp ? ceil_div(teams, kWarpTeams) : teams)), dim3(s.threads), 0,
               (cudaStream_t)stream, pdl, 1, a);
  }
  if (e == cudaSuccess && planes > 0) {
    float *out[3] = {nullptr, nullptr, nullptr};
    int k = 0;
    if (w_pre) out[k++] = dw_pre;
    if (w_post) out[k++] = dw_post;
    if (channel_gate) out[k++] = static_cast<float *>(dgate);
    e = launch(norm_colsum_kernel, dim3(static_cast<unsigned>(ceil_div(static_cast<int64_t>(planes) * n, 32))), dim3(32, 32), 0,
               (cudaStream_t)stream, pdl, 1, (const float *)workspace, teams, planes, static_cast<int>(n), out[0], out[1], out[2]);
  }
  return check_launch(e, name);
}
