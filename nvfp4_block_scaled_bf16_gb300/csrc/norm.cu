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
// Every kernel reads each input once: they are bound by memory for many rows and by latency for few.
// A team (a warp up to 512 channels, otherwise a block) owns a row; a thread holds 8 * VPT of its channels.
//   - norm_kernel, norm_grad_kernel: the row's loads go straight to registers, one team per row;
//   - norm_ring_kernel, norm_grad_ring_kernel, for many aligned rows of more than 512 channels: resident
//     blocks walk the rows, which bulk copies bring ahead into a ring of shared memory, with one barrier a
//     row; registers alone cannot hold enough loads in flight across a row's reductions.
#include <cuda_bf16.h>

#include <type_traits>

#include "host.h"
#include "ptx.cuh"

namespace nvfp4 {
namespace {

constexpr int kSiteRing = 7;  // wait site recorded in the status word (after the GEMM's, gemm.cuh)
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

// A row of an operand.  Channels past n read as zero, and so add nothing to any sum below.
// AHEAD: load() loads, late() converts.  A kernel calls load() for every operand first: with load and
// conversion together in each operand's branch, every operand waited for memory on its own (backward,
// 2048 x 2047: 63 -> 35 us; forward, 4096 x 328: 8.2 -> 6.2 us).  Otherwise load() only notes the address and
// early() does both: single channels in flight cost a register each (kernels say where that is too many).
template <int VPT, bool VEC, bool AHEAD, typename T>
struct Row {
  static constexpr int kWords = VEC ? VPT * static_cast<int>(sizeof(T)) / 2 : 1;
  static constexpr int kSingles = VEC ? 1 : 8 * VPT;
  uint4 w[kWords];
  T s[kSingles];
  const T *at;
  bool is;
  // given: whether there is such an operand; one that is not there reads as zero.
  __device__ __forceinline__ void load(bool given, const T *row, int t, int ts, int n) {
    at = row;
    is = given;
    if constexpr (AHEAD) fetch(t, ts, n);
  }
  __device__ __forceinline__ void early(float (&f)[8 * VPT], int t, int ts, int n) {
    if constexpr (!AHEAD) {
      fetch(t, ts, n);
      convert(f);
    }
  }
  __device__ __forceinline__ void late(float (&f)[8 * VPT]) const {
    if constexpr (AHEAD) convert(f);
  }

 private:
  __device__ __forceinline__ void zero() {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < kSingles; ++i) s[i] = T(0.0f);
    }
  }
  __device__ __forceinline__ void fetch(int t, int ts, int n) {
    zero();
    if (!is) return;
    if constexpr (VEC) {
      constexpr int W = kWords / VPT;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = (v * ts + t) * 8;
        if (c < n)
#pragma unroll
          for (int k = 0; k < W; ++k) w[v * W + k] = reinterpret_cast<const uint4 *>(at + c)[k];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kSingles; ++i) {
        const int c = i * ts + t;
        if (c < n) s[i] = at[c];
      }
    }
  }
  __device__ __forceinline__ void convert(float (&f)[8 * VPT]) const {
    if constexpr (VEC) {
      constexpr int W = kWords / VPT;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
          const uint4 q = w[v * W + k];
          const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
              f[8 * v + 4 * k + i] = __uint_as_float(u[i]);
            } else {
              f[8 * v + 2 * i] = __uint_as_float(u[i] << 16);
              f[8 * v + 2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
            }
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kSingles; ++i) f[i] = to_f32(s[i]);
    }
  }
};
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

// NVFP4 of channels already rounded to bf16, eight from c on in each lane: a 16-channel block is the 8 channels of two neighbouring
// threads, and eight threads gather the four scale bytes of a 32-bit word of the 128x4 layout.
// Every lane of the warp takes part; channels past n (whole blocks) get zero scales.
__device__ __forceinline__ void quantize8(const NormArgs &p, const float *f, float gs, int64_t row, int c) {
  float amax = 0.0f, y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  uint32_t code = 0;
  const float inv = nvfp4_block_scale(amax, gs, code);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(f[i], inv);
  if (c < p.n) *reinterpret_cast<uint32_t *>(p.q + row * (p.n >> 1) + (c >> 1)) = e2m1x8(y);
  else code = 0;
  const uint32_t b1 = __shfl_down_sync(0xFFFFFFFFu, code, 2);
  const uint32_t b2 = __shfl_down_sync(0xFFFFFFFFu, code, 4);
  const uint32_t b3 = __shfl_down_sync(0xFFFFFFFFu, code, 6);
  const int j = c >> 4;  // scale column
  if ((threadIdx.x & 7) == 0 && j < p.cp)
    *reinterpret_cast<uint32_t *>(p.sf + ((row >> 7) * (p.cp >> 2) + (j >> 2)) * 512 + (row & 31) * 16 +
                                  ((row >> 5) & 3) * 4) = code | (b1 << 8) | (b2 << 16) | (b3 << 24);
}
template <int VPT>
__device__ __forceinline__ void quantize_row(const NormArgs &p, const float (&f)[8 * VPT], int64_t row, int t, int ts) {
  const float gs = __ldg(p.gs);
#pragma unroll
  for (int v = 0; v < VPT; ++v) quantize8(p, f + 8 * v, gs, row, (v * ts + t) * 8);
}

// Zeroes the scale rows between m and the next multiple of 128 (block `block` of `blocks`).
__device__ __forceinline__ void zero_pad_rows(const NormArgs &p, unsigned int block, unsigned int blocks) {
  const int64_t words = ((p.m + 127) / 128 * 128 - p.m) * (p.cp >> 2);
  const int64_t stride = static_cast<int64_t>(blocks) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(block) * blockDim.x + threadIdx.x; i < words; i += stride) {
    const int64_t row = p.m + i / (p.cp >> 2), jt = i % (p.cp >> 2);
    *reinterpret_cast<uint32_t *>(p.sf + ((row >> 7) * (p.cp >> 2) + jt) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4) = 0u;
  }
}

// Blocks [0, row_blocks) hold the rows; with NVFP4 output the blocks after them zero the scale rows
// between m and the next multiple of 128.
// MAXT: threads of the largest block it is launched with (512, 768 or 1024: 128, 80 or 64 registers).
// The one block an SM is spelled out for 1024: without it the compiler gave the widest rows 32 registers
// (512 x 32768 forward 141 -> 65 us, 1024 x 8200 backward 162 -> 96, 512 x 32768 backward 567 -> 363).
template <typename XT, int VPT, bool VEC, bool WARP, bool QUANT, int MAXT>
__global__ void __launch_bounds__(WARP ? 32 * kWarpTeams : MAXT, MAXT == 1024 ? 1 : 0)
    norm_kernel(const NormArgs p, unsigned int row_blocks) {
  __shared__ float s_buf[2][1][32];
  // The next kernel may launch now: it waits for this grid before it reads what is written here.
  pdl_trigger();
  pdl_wait();
  if (QUANT && blockIdx.x >= row_blocks) {
    zero_pad_rows(p, blockIdx.x - row_blocks, gridDim.x - row_blocks);
    return;
  }
  const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpTeams + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= p.m) return;
  const int t = WARP ? threadIdx.x & 31 : threadIdx.x, ts = WARP ? 32 : blockDim.x;
  constexpr int E = 8 * VPT;
  TeamSum<1> team{s_buf};
  const float inv_n = 1.0f / static_cast<float>(p.n);
  // (loaded ahead, a block's rows of single channels and rows of four vectors a thread were slower: 1024 x 8191
  // 39 -> 46 us, 8 x 16385 22 -> 44, 512 x 32768 66 -> 92; registers again)
  constexpr bool AHEAD = (VEC || WARP) && VPT < 4;
  using Bf16Row = Row<VPT, VEC, AHEAD, __nv_bfloat16>;
  float r[E], w[E];
  Row<VPT, VEC, AHEAD, XT> rx;
  Bf16Row ry, rw, rwp, rg;
  rx.load(true, static_cast<const XT *>(p.x) + row * p.ldx, t, ts, p.n);
  ry.load(p.y != nullptr, p.y + row * p.ldy, t, ts, p.n);
  rw.load(p.w_pre != nullptr, p.w_pre, t, ts, p.n);
  rwp.load(p.w_post != nullptr, p.w_post, t, ts, p.n);
  rg.load(p.gate != nullptr, p.gate + row * p.ldg, t, ts, p.n);
  rx.early(r, t, ts, p.n), rx.late(r);
  if (p.y) {
    float y[E];
    ry.early(y, t, ts, p.n), ry.late(y);
    rw.early(w, t, ts, p.n);
    if (p.w_post) {
      float wp[E];
      rwp.early(wp, t, ts, p.n);
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < E; ++i) s[0] += y[i] * y[i];
      team.template sum<WARP>(s);
      const float rstd = rsqrtf(s[0] * inv_n + p.eps);
      rwp.late(wp);
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] = y[i] * rstd * (p.offset + wp[i]);
    }
    if (p.gate) {
      float g[E];
      rg.early(g, t, ts, p.n), rg.late(g);
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] *= g[i];
    }
#pragma unroll
    for (int i = 0; i < E; ++i) r[i] = r[i] + p.scale * y[i];
    store_row<VPT, VEC>(static_cast<XT *>(p.x_out) + row * p.ldxo, r, t, ts, p.n);
  } else {
    rw.early(w, t, ts, p.n);
  }
  if (!p.w_pre) return;
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < E; ++i) s[0] += r[i] * r[i];
  team.template sum<WARP>(s);
  const float rstd = rsqrtf(s[0] * inv_n + p.eps);
  rw.late(w);
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

// Two fp32 values in a register pair: Blackwell's packed arithmetic rounds each half as the scalar
// instruction would, at half the instructions.  The ring kernels are written in it: with scalar
// arithmetic the 4096 x 7168 forward pass spent 36 instructions a channel and was bound by their issue.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void halves(F2 a, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v)); }
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float sum(F2 a) {
  float lo, hi;
  halves(a, lo, hi);
  return lo + hi;
}
// Pair i of eight bf16 channels.
__device__ __forceinline__ F2 pair(const uint4 &q, int i) {
  const uint32_t w = i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// Eight channels as four pairs, from and to memory.
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, F2 *f) {
  const uint4 q = *reinterpret_cast<const uint4 *>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pair(q, i);
}
__device__ __forceinline__ void load4(const float *p, F2 *f) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(p)[0], b = reinterpret_cast<const ulonglong2 *>(p)[1];
  f[0].v = a.x, f[1].v = a.y, f[2].v = b.x, f[3].v = b.y;
}
__device__ __forceinline__ uint32_t pack(F2 a) {
  float lo, hi;
  halves(a, lo, hi);
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const F2 *f) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack(f[0]), pack(f[1]), pack(f[2]), pack(f[3]));
}
__device__ __forceinline__ void store4(float *p, const F2 *f) {
  reinterpret_cast<ulonglong2 *>(p)[0] = make_ulonglong2(f[0].v, f[1].v);
  reinterpret_cast<ulonglong2 *>(p)[1] = make_ulonglong2(f[2].v, f[3].v);
}

// A row's operands as they land in one slot of the ring, each 16-byte aligned; 0 bytes: absent.
struct Slot {
  int bytes[5], offset[5], size;
};
template <int N>
Slot slot_of(const int (&bytes)[N]) {
  Slot s{};
  for (int i = 0; i < N; ++i) {
    s.bytes[i] = bytes[i];
    s.offset[i] = s.size;
    s.size += bytes[i];
  }
  return s;
}
struct RingArgs {
  int slots;
  Slot slot;
  unsigned int *status;
  long long wait_limit;
};

constexpr int kMaxSlots = 4;
constexpr int kRingHead = 128;  // shared memory ahead of the slots: a barrier per slot, the abort flag

// The ring of one block: its rows are first, first + step, ..., row i of them in slot i % slots.  An operand's
// copy goes out from lane 0 of a warp of its own (a copy costs the thread that issues it about 100 cycles,
// which the block's next barrier would wait for); a slot's barrier collects one arrival per operand.
struct Ring {
  uint64_t *full;
  volatile int *abort;
  uint8_t *data;
  const RingArgs &a;
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ Ring(uint8_t *smem, const RingArgs &args)
      : full(reinterpret_cast<uint64_t *>(smem)), abort(reinterpret_cast<volatile int *>(smem + 8 * kMaxSlots)),
        data(smem + kRingHead), a(args) {
    if (threadIdx.x == 0) {
      int operands = 0;
      for (int o = 0; o < 5; ++o) operands += a.slot.bytes[o] > 0;
      for (int i = 0; i < a.slots; ++i) mbar_init(smem_u32(&full[i]), operands);
      *abort = 0;
      fence_barrier_init();
    }
    __syncthreads();
  }
  // src(operand): where the row begins
  template <class Src>
  __device__ __forceinline__ void fill(int to, Src &&src) const {
    if ((threadIdx.x & 31) != 0) return;
    for (int o = threadIdx.x >> 5; o < 5; o += blockDim.x >> 5) {
      const int bytes = a.slot.bytes[o];
      if (!bytes) continue;
      mbar_arrive_expect_tx(smem_u32(&full[to]), bytes);
      bulk_load(smem_u32(data + to * a.slot.size) + a.slot.offset[o], src(o), bytes, smem_u32(&full[to]));
    }
  }
  // Waits for the slot; one that gives up sets the abort flag, which the block reads behind its next barrier.
  __device__ __forceinline__ void wait(int i, uint32_t parity) const {
    const WaitCtl wc{a.wait_limit, abort, a.status};
    mbar_wait(smem_u32(&full[i]), parity, wc, kSiteRing);
  }
  template <typename T>
  __device__ __forceinline__ const T *operand(int i, int o) const {
    return reinterpret_cast<const T *>(data + i * a.slot.size + a.slot.offset[o]);
  }
  __device__ __forceinline__ int next_slot() const { return slot + 1 == a.slots ? 0 : slot + 1; }
  __device__ __forceinline__ uint32_t next_phase() const { return slot + 1 == a.slots ? phase ^ 1 : phase; }
  __device__ __forceinline__ void advance() {
    phase = next_phase();
    slot = next_slot();
  }
  // After a wait gave up: thread 0 waits, again with a limit, for the copies still in flight, so that
  // none lands after the block is gone.
  __device__ void drain() {
    if (threadIdx.x != 0) return;
    for (int n = 0; n < a.slots; ++n) {
      const long long t0 = clock64();
      while (!mbar_try_wait(smem_u32(&full[slot]), phase) && clock64() - t0 < a.wait_limit) {
      }
      advance();
    }
  }
};

// norm_kernel for many rows (see the head of this file).  The sums of r^2 of a row
// and of y^2 of the row after it share a barrier.  A thread keeps its channels' factors in fp32:
// scale * gate * (offset + w_post) of y and offset + w_pre.
// Measured at 4096 x 7168, cold L2: 48 to 49 us for 235 MB, where 34.9 us is the measured copy rate and 37 us
// what a kernel takes that only reads two such arrays and writes two.  Against it, the same ring with two
// barriers a row and the copies issued by one computing thread took 54 us, a warp per row 74 us (too few
// warps fit beside the rows), plain loads 59 us, one more warp for the copies 52 us.  What is left is
// the latency of a row's chain (slot, sums, barrier, stores) that two blocks do not hide entirely: without
// the stores of x_out it takes 43.5 us, with 2 slots instead of 3 49.7 us.
template <typename XT, int VPT, bool QUANT, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_ring_kernel(const NormArgs p, const RingArgs ra) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_sum[2][2][32];  // [value][warp]; warps that are not there add zero
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, ts = blockDim.x;
  for (int i = t; i < 2 * 2 * 32; i += blockDim.x) (&s_sum[0][0][0])[i] = 0.0f;
  Ring ring(smem, ra);
  const int64_t first = blockIdx.x, step = gridDim.x;
  auto fill = [&](int to, int64_t row) {
    ring.fill(to, [&](int o) -> const void * {
      if (o == 0) return static_cast<const XT *>(p.x) + row * p.ldx;
      return o == 1 ? p.y + row * p.ldy : p.gate + row * p.ldg;
    });
  };
  for (int i = 0; i < ra.slots && first + i * step < p.m; ++i) fill(i, first + i * step);
  const bool token_gate = p.gate && p.ldg != 0;
  const F2 zero = f2(0.0f), offset = f2(p.offset);
  constexpr int P = 4 * VPT;  // pairs a thread holds
  F2 factor[P], pre[P];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (v * ts + t) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) factor[4 * v + i] = f2(p.scale), pre[4 * v + i] = zero;
    if (c >= p.n) continue;
    F2 w[4];
    if (p.w_post) {
      load4(p.w_post + c, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) factor[4 * v + i] = factor[4 * v + i] * (offset + w[i]);
    }
    if (p.gate && !token_gate) {
      load4(p.gate + c, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) factor[4 * v + i] = factor[4 * v + i] * w[i];
    }
    if (p.w_pre) {
      load4(p.w_pre + c, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) pre[4 * v + i] = offset + w[i];
    }
  }
  const float inv_n = 1.0f / static_cast<float>(p.n), gs = QUANT ? __ldg(p.gs) : 0.0f;
  const bool norm_y = p.y && p.w_post;
  // sum of y^2 of the row in slot i
  auto squares = [&](int i) {
    F2 q = zero, y[4];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * ts + t) * 8;
      if (c >= p.n) continue;
      load4(ring.operand<__nv_bfloat16>(i, 1) + c, y);
#pragma unroll
      for (int k = 0; k < 4; ++k) q = fma(y[k], y[k], q);
    }
    return sum(q);
  };
  int buf = 0;
  // block sums of a and b, in a fixed order: the first shuffle leaves a to the lower half warp and b to the
  // upper.  False: a wait gave up.
  auto block_sums = [&](float &a, float &b) {
    float s = lane < 16 ? a : b;
    s += __shfl_xor_sync(0xFFFFFFFFu, lane < 16 ? b : a, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s_sum[buf][lane >> 4][warp] = s;  // (by every lane of the half: under a test of lane & 15 the compiler takes
                                      // lane >> 4 for lane / 16 without its remainder further down, too)
    __syncthreads();
    s = s_sum[buf][lane >> 4][lane & 15] + s_sum[buf][lane >> 4][(lane & 15) + 16];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    a = __shfl_sync(0xFFFFFFFFu, s, 0);
    b = __shfl_sync(0xFFFFFFFFu, s, 16);
    buf ^= 1;  // (written again only after the next sums' barrier)
    return *ring.abort == 0;
  };
  float ry = 1.0f;
  bool ok = true;
  if (norm_y && first < p.m) {
    ring.wait(0, 0);
    float a = 0.0f, b = squares(0);
    ok = block_sums(a, b);
    ry = rsqrtf(b * inv_n + p.eps);
  }
  for (int64_t row = first; ok && row < p.m; row += step) {
    ring.wait(ring.slot, ring.phase);
    F2 r[P], q = zero;
    const F2 f = f2(ry);
    float yy = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * ts + t) * 8;
      if (c >= p.n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[4 * v + i] = zero;
        continue;
      }
      load4(ring.operand<XT>(ring.slot, 0) + c, r + 4 * v);
      if (p.y) {
        F2 y[4];
        load4(ring.operand<__nv_bfloat16>(ring.slot, 1) + c, y);
        if (token_gate) {
          F2 g[4];
          load4(ring.operand<__nv_bfloat16>(ring.slot, 2) + c, g);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = y[i] * g[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) r[4 * v + i] = fma(y[i] * factor[4 * v + i], f, r[4 * v + i]);
        store4(static_cast<XT *>(p.x_out) + row * p.ldxo + c, r + 4 * v);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) q = fma(r[4 * v + i], r[4 * v + i], q);
    }
    float rr = sum(q);
    if (norm_y && row + step < p.m) {
      ring.wait(ring.next_slot(), ring.next_phase());
      yy = squares(ring.next_slot());
    }
    ok = block_sums(rr, yy);
    if (!ok) break;
    // every thread has read this row's slot
    if (row + ra.slots * step < p.m) fill(ring.slot, row + ra.slots * step);
    ry = norm_y ? rsqrtf(yy * inv_n + p.eps) : 1.0f;
    if (p.w_pre) {
      const F2 rstd = f2(rsqrtf(rr * inv_n + p.eps));
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = (v * ts + t) * 8;
        F2 *h = r + 4 * v;
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = h[i] * rstd * pre[4 * v + i];
        if constexpr (QUANT) {
          float q8[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w = pack(h[i]);  // rounded to bf16, then widened again
            q8[2 * i] = __uint_as_float(w << 16);
            q8[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
          }
          quantize8(p, q8, gs, row, c);
        } else if (c < p.n) {
          store4(p.h + row * p.ldh + c, h);
        }
      }
    }
    ring.advance();
  }
  if (!ok) ring.drain();
  if constexpr (QUANT) zero_pad_rows(p, blockIdx.x, gridDim.x);
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
__global__ void __launch_bounds__(WARP ? 32 * kWarpTeams : MAXT, MAXT > 512 ? 1 : 0)
    norm_grad_kernel(const NormGradArgs p) {
  __shared__ float s_buf3[2][3][32];
  __shared__ float s_buf1[2][1][32];
  pdl_trigger();
  pdl_wait();
  const int teamid = WARP ? blockIdx.x * kWarpTeams + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && teamid >= p.teams) return;
  const int t = WARP ? threadIdx.x & 31 : threadIdx.x, ts = WARP ? 32 : blockDim.x;
  constexpr int E = 8 * VPT;
  // (1024 threads have 64 registers each; loaded ahead: 1024 x 8191 94 -> 111 us, 1 x 7168 17 -> 23)
  constexpr bool AHEAD = MAXT < 1024;
  using Bf16Row = Row<VPT, VEC, AHEAD, __nv_bfloat16>;
  TeamSum<3> team3{s_buf3};
  TeamSum<1> team1{s_buf1};
  const float inv_n = 1.0f / static_cast<float>(p.n);
  float aw[E], ap[E], ag[E];
#pragma unroll
  for (int i = 0; i < E; ++i) aw[i] = ap[i] = ag[i] = 0.0f;
  for (int64_t row = teamid; row < p.m; row += p.teams) {
    float r[E], d[E], g[E], y[E];
    Row<VPT, VEC, AHEAD, XT> rr, rdr;
    Bf16Row rd, ry, rw, rwp, rg;
    rr.load(true, static_cast<const XT *>(p.r) + row * p.ldr, t, ts, p.n);
    rd.load(p.dh != nullptr, p.dh + row * p.lddh, t, ts, p.n);
    rdr.load(p.dr != nullptr, static_cast<const XT *>(p.dr) + row * p.lddr, t, ts, p.n);
    ry.load(p.y != nullptr, p.y + row * p.ldy, t, ts, p.n);
    rw.load(p.dh != nullptr, p.w_pre, t, ts, p.n);
    rwp.load(p.w_post != nullptr, p.w_post, t, ts, p.n);
    rg.load(p.gate != nullptr, p.gate + row * p.ldg, t, ts, p.n);
    rr.early(r, t, ts, p.n), rd.early(d, t, ts, p.n), rdr.early(g, t, ts, p.n), ry.early(y, t, ts, p.n);
    rr.late(r), rd.late(d), rdr.late(g), ry.late(y);
    // sums of r^2, of (dh w) r and of y^2 in one go: mean(d xn) = rstd * sum(d r) / n
    float s[3] = {0.0f, 0.0f, 0.0f};
    {
      float w[E];
      rw.early(w, t, ts, p.n), rw.late(w);
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
      rwp.early(wp, t, ts, p.n), rwp.late(wp);
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
      rg.early(d, t, ts, p.n), rg.late(d);
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

// norm_grad_kernel for many rows (see the head of this file).  A row needs one reduction only: dy's mean is
// linear in the gradient of r, so with u = gate * (offset + w_post) the sums
//   r^2, (dh w) r, y^2,  A = u y dr,  B = u y dh w,  C = u y r       (w = offset + w_pre)
// give it as scale * rstd_y / n * (A + rstd_r B - rstd_r^2 mean C), mean = rstd_r sum((dh w) r) / n.
// Warp shuffles that halve the values a lane carries, then the lanes, take 9 shuffles for all six.  A row
// is read from its slot twice, before and after the block's barrier; the barrier of row i also says that
// row i - 1 is done with, so its slot is filled again behind it.
template <typename XT, int VPT, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_grad_ring_kernel(const NormGradArgs p, const RingArgs ra) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float s_sum[2][8][32];  // [value][warp]; warps that are not there add zero
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, ts = blockDim.x;
  for (int i = t; i < 2 * 8 * 32; i += ts) (&s_sum[0][0][0])[i] = 0.0f;
  Ring ring(smem, ra);
  const int64_t first = blockIdx.x, step = gridDim.x;
  auto fill = [&](int to, int64_t row) {
    ring.fill(to, [&](int o) -> const void * {
      if (o == 0) return static_cast<const XT *>(p.r) + row * p.ldr;
      if (o == 1) return p.dh + row * p.lddh;
      if (o == 2) return static_cast<const XT *>(p.dr) + row * p.lddr;
      return o == 3 ? p.y + row * p.ldy : p.gate + row * p.ldg;
    });
  };
  for (int i = 0; i < ra.slots && first + i * step < p.m; ++i) fill(i, first + i * step);
  const float inv_n = 1.0f / static_cast<float>(p.n);
  uint4 w_pre[VPT], w_post[VPT], gate[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (v * ts + t) * 8;
    w_pre[v] = w_post[v] = gate[v] = make_uint4(0u, 0u, 0u, 0u);
    if (c < p.n) {
      if (p.w_pre) w_pre[v] = *reinterpret_cast<const uint4 *>(p.w_pre + c);
      if (p.w_post) w_post[v] = *reinterpret_cast<const uint4 *>(p.w_post + c);
      if (p.gate && p.ldg == 0) gate[v] = *reinterpret_cast<const uint4 *>(p.gate + c);
    }
  }
  const F2 offset = f2(p.offset), zero = f2(0.0f), one = f2(1.0f);
  const bool token_gate = p.gate && p.ldg != 0;
  constexpr int P = 4 * VPT;  // pairs a thread holds
  F2 aw[P], ap[P], ag[P];
#pragma unroll
  for (int i = 0; i < P; ++i) aw[i] = ap[i] = ag[i] = zero;
  int buf = 0;
  bool gone = false;
  for (int64_t row = first; row < p.m; row += step) {
    ring.wait(ring.slot, ring.phase);
    const XT *in_r = ring.operand<XT>(ring.slot, 0), *in_g = ring.operand<XT>(ring.slot, 2);
    const __nv_bfloat16 *in_d = ring.operand<__nv_bfloat16>(ring.slot, 1), *in_y = ring.operand<__nv_bfloat16>(ring.slot, 3),
                        *in_gate = ring.operand<__nv_bfloat16>(ring.slot, 4);
    F2 q[6] = {zero, zero, zero, zero, zero, zero};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * ts + t) * 8;
      if (c >= p.n) continue;
      F2 r[4], dw[4], u[4];
      load4(in_r + c, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) dw[i] = zero;
      if (p.dh) {
        load4(in_d + c, dw);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dw[i] = dw[i] * (offset + pair(w_pre[v], i));
          q[0] = fma(r[i], r[i], q[0]);
          q[1] = fma(dw[i], r[i], q[1]);
        }
      }
      if (p.w_post) {
        load4(in_y + c, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          q[2] = fma(u[i], u[i], q[2]);
          u[i] = u[i] * (offset + pair(w_post[v], i));
        }
        if (p.gate) {
          if (token_gate) gate[v] = *reinterpret_cast<const uint4 *>(in_gate + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) u[i] = u[i] * pair(gate[v], i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          q[4] = fma(u[i], dw[i], q[4]);
          q[5] = fma(u[i], r[i], q[5]);
        }
        if (p.dr) {
          load4(in_g + c, r);
#pragma unroll
          for (int i = 0; i < 4; ++i) q[3] = fma(u[i], r[i], q[3]);
        }
      }
    }
    // six sums over the warp: each step halves the values a lane carries (then the lanes)
    float s[8] = {sum(q[0]), sum(q[1]), sum(q[2]), sum(q[3]), sum(q[4]), sum(q[5]), 0.0f, 0.0f};
#pragma unroll
    for (int k = 4, o = 16; k > 0; k >>= 1, o >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < k; ++i) {
        const float keep = up ? s[i + k] : s[i], give = up ? s[i] : s[i + k];
        s[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
      }
    }
    s[0] += __shfl_xor_sync(0xFFFFFFFFu, s[0], 2);
    s[0] += __shfl_xor_sync(0xFFFFFFFFu, s[0], 1);
    // lanes 4 i .. 4 i + 3 hold value ((i >> 2) & 1) * 4 + ((i >> 1) & 1) * 2 + (i & 1)  =  i
    s_sum[buf][lane >> 2][warp] = s[0];  // (by all four: see norm_ring_kernel)
    __syncthreads();
    if (*ring.abort) {
      gone = true;
      break;
    }
    // every thread has done with the row before this one: its slot is free
    if (row != first && row + (ra.slots - 1) * step < p.m)
      fill(ring.slot == 0 ? ra.slots - 1 : ring.slot - 1, row + (ra.slots - 1) * step);
    float tot;
    {
      const float4 a = *reinterpret_cast<const float4 *>(&s_sum[buf][lane >> 2][(lane & 3) * 8]);
      const float4 b = *reinterpret_cast<const float4 *>(&s_sum[buf][lane >> 2][(lane & 3) * 8 + 4]);
      tot = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
      tot += __shfl_xor_sync(0xFFFFFFFFu, tot, 2);
      tot += __shfl_xor_sync(0xFFFFFFFFu, tot, 1);
    }
    buf ^= 1;  // (written again only after the next row's barrier)
    float v6[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) v6[i] = __shfl_sync(0xFFFFFFFFu, tot, 4 * i);
    const float rx1 = rsqrtf(v6[0] * inv_n + p.eps), mean1 = v6[1] * rx1 * inv_n;
    const float ry1 = p.w_post ? rsqrtf(v6[2] * inv_n + p.eps) : 1.0f;
    // without w_post dy has no mean; without dh the stream has no part in it (and rx1 and mean1 mean nothing: r^2
    // is not added up, so with eps = 0 they are inf and NaN)
    float dot = v6[3];
    if (p.dh) dot = v6[3] + rx1 * v6[4] - rx1 * rx1 * mean1 * v6[5];
    const float e1 = p.w_post ? p.scale * ry1 * inv_n * dot : 0.0f;
    const F2 rx = f2(rx1), neg_mean = f2(-mean1), ry = f2(ry1), neg_e = f2(-e1), scale = f2(p.scale);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * ts + t) * 8;
      if (c >= p.n) continue;
      F2 g[4], a[4], b[4];
      if (p.dr) {
        load4(in_g + c, g);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = zero;
      }
      if (p.dh) {
        load4(in_r + c, a);
        load4(in_d + c, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 xn = a[i] * rx;
          aw[4 * v + i] = fma(b[i], xn, aw[4 * v + i]);
          g[i] = fma(rx, fma(xn, neg_mean, b[i] * (offset + pair(w_pre[v], i))), g[i]);
        }
      }
      store4(static_cast<XT *>(p.dx) + row * p.lddx + c, g);
      if (!p.y) continue;
      load4(in_y + c, a);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = a[i] * ry;      // yn
        g[i] = g[i] * scale;
        b[i] = p.w_post ? offset + pair(w_post[v], i) : one;
      }
      if (p.gate) {
        F2 d[4];
        if (token_gate) gate[v] = *reinterpret_cast<const uint4 *>(in_gate + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d[i] = g[i] * a[i] * b[i];
          g[i] = g[i] * pair(gate[v], i);
        }
        if (token_gate) {
          store4(p.dgate + row * p.lddg + c, d);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) ag[4 * v + i] = ag[4 * v + i] + d[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ap[4 * v + i] = fma(g[i], a[i], ap[4 * v + i]);
        if (p.w_post) g[i] = ry * fma(a[i], neg_e, g[i] * b[i]);  // (otherwise dy does not depend on y)
      }
      store4(p.dy + row * p.lddy + c, g);
    }
    ring.advance();
  }
  if (gone) {
    ring.drain();
    return;
  }
  auto store_sums = [&](float *part, const F2 *f) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * ts + t) * 8;
      if (c < p.n) store4(part + c, f + 4 * v);
    }
  };
  float *part = p.part + static_cast<int64_t>(blockIdx.x) * p.planes * p.n;
  if (p.dh) {
    store_sums(part, aw);
    part += p.n;
  }
  if (p.y && p.w_post) {
    store_sums(part, ap);
    part += p.n;
  }
  if (p.y && p.gate && p.ldg == 0) store_sums(part, ag);
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
  if constexpr (MAXT > 512) {  // (more than 512 threads of two vectors each come before four vectors)
    if (vpt == 4) return norm_kernel<XT, 4, VEC, false, QUANT, MAXT>;
    if (vpt == 2) return norm_kernel<XT, 2, VEC, false, QUANT, MAXT>;
  } else if constexpr (VEC && sizeof(XT) == 4) {  // (two vectors: forward_vpt)
    if (vpt == 2) return norm_kernel<XT, 2, VEC, false, QUANT, MAXT>;
  }
  return norm_kernel<XT, 1, VEC, false, QUANT, MAXT>;
}
template <typename XT, bool VEC, bool QUANT>
auto forward_kernel(const Shape &s) {
  if (s.warp) return s.vpt == 1 ? norm_kernel<XT, 1, VEC, true, QUANT, 512> : norm_kernel<XT, 2, VEC, true, QUANT, 512>;
  return s.threads <= 512 ? forward_block<XT, VEC, QUANT, 512>(s.vpt) : forward_block<XT, VEC, QUANT, 1024>(s.vpt);
}
template <typename XT, bool VEC>
auto backward_kernel(const Shape &s) {
  if (s.warp) return s.vpt == 1 ? norm_grad_kernel<XT, 1, VEC, true, 512> : norm_grad_kernel<XT, 2, VEC, true, 512>;
  if (s.threads <= 512) return norm_grad_kernel<XT, 1, VEC, false, 512>;  // (one vector a thread up to 1024 threads)
  // (80 registers instead of 64: 2048 x 4099 126 -> 98 us)
  if (s.threads <= 768 && s.vpt == 1) return norm_grad_kernel<XT, 1, VEC, false, 768>;
  return s.vpt == 1 ? norm_grad_kernel<XT, 1, VEC, false, 1024>
                    : (s.vpt == 2 ? norm_grad_kernel<XT, 2, VEC, false, 1024> : norm_grad_kernel<XT, 4, VEC, false, 1024>);
}

// Teams of the backward pass: as many blocks as an SM holds at up to 104 registers a thread, each with a
// row of its own (two whatever their size: 4096 x 723 82 us, 62 so); more than two of them only where each
// keeps two rows (600 x 720 with a row a block 12.4 us instead of 10.3: its sums are written and read for
// one row).  (Fixed per shape and device, so that the order of the column sums is too.)
int grad_teams(int64_t m, const Shape &s, int sm_count) {
  const int64_t per_sm = s.warp ? 4 * kWarpTeams : (s.threads < 630 ? 630 / s.threads : 1);
  int64_t cap = per_sm * sm_count;
  if (!s.warp && cap > 2 * sm_count) cap = m / 2 < 2 * sm_count ? 2 * sm_count : (m / 2 < cap ? m / 2 : cap);
  return static_cast<int>(m < cap ? m : cap);
}

constexpr int kSmemBudget = 226 * 1024;  // dynamic shared memory of all blocks of an SM together

// Ring launches: blocks of `threads` threads of `vpt` vectors each, per_sm of them an SM.  Taken from four
// rows an SM on (fewer: the plain kernels start sooner), for 513 to 8192 channels.
struct RingShape {
  bool use;
  int vpt, threads, per_sm, slots;
};
// Two slots for each block of an SM, or no ring.  All widths have them but the widest rows of an fp32 stream with a
// gate per token (a slot of x, y and gate is 8 bytes a channel, with dh and dx_out 14): 7040 to 7168 channels
// forward, where two blocks share the SM, and from 8152 on backward.  (Forward it costs nothing: 1024 x 7168 23.8 us
// by norm_kernel, 1024 x 7032 26.6 by the ring.)
RingShape ring_slots(RingShape s, int slot) {
  s.slots = (kSmemBudget / s.per_sm - kRingHead - 3 * 1024) / slot;
  if (s.slots > kMaxSlots) s.slots = kMaxSlots;
  s.use = s.slots >= 2;
  return s;
}
// n_pad: channels the NVFP4 scale columns need.  One vector a thread up to 4096 channels (64 registers), two
// above (half the warps share a row's fixed costs: 4096 x 7168 49.6 -> 47.6 us), two blocks an SM up to 7168.
RingShape forward_ring_shape(int64_t m, int64_t n_pad, int slot, int sm_count) {
  RingShape s{};
  const int nv = static_cast<int>(ceil_div(n_pad, 8));
  if (m < 4LL * sm_count || nv <= 64 || nv > 1024) return s;
  s.vpt = nv > 512 ? 2 : 1;
  s.threads = static_cast<int>(round_up(ceil_div(nv, s.vpt), 32));
  s.per_sm = s.vpt == 2 ? (s.threads <= 448 ? 2 : 1) : s.threads <= 256 ? 4 : 2;
  return ring_slots(s, slot);
}
// One vector a thread up to 4096 channels, two above; 128 registers a thread.
RingShape backward_ring_shape(int64_t m, int64_t n, int slot, int sm_count) {
  RingShape s{};
  const int nv = static_cast<int>(ceil_div(n, 8));
  if (m < 4LL * sm_count || nv <= 64 || nv > 1024) return s;
  s.vpt = nv > 512 ? 2 : 1;
  s.threads = static_cast<int>(round_up(ceil_div(nv, s.vpt), 32));
  s.per_sm = s.threads <= 128 ? 4 : s.threads <= 256 ? 2 : 1;
  return ring_slots(s, slot);
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
  if (flags & ~(uint32_t)(NVFP4_FLAG_PDL | NVFP4_FLAG_DEBUG_TIMEOUT)) return fail(NVFP4_ERR_INVALID_ARG, "%s: unknown flags 0x%x", name, flags);
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

// Launches the forward pass as a ring where that pays; false: it does not.
template <bool QUANT>
static bool forward_ring(const NormArgs &a, bool f32, bool pdl, cudaStream_t stream, const DeviceInfo &dev, uint32_t flags,
                         nvfp4_status_t *st, const char *name) {
  const int n = a.n, xe = f32 ? 4 : 2;
  const int bytes[3] = {n * xe, a.y ? n * 2 : 0, a.y && a.gate && a.ldg != 0 ? n * 2 : 0};
  const Slot slot = slot_of(bytes);
  const RingShape s = forward_ring_shape(a.m, QUANT ? a.cp * 16 : n, slot.size, dev.sm_count);
  if (!s.use) return false;
  const RingArgs ra{s.slots, slot, dev.status, wait_limit(flags)};
  auto pick = [&](auto *x) {
    using XT = std::remove_pointer_t<decltype(x)>;
    if (s.vpt == 2) return s.threads <= 448 ? norm_ring_kernel<XT, 2, QUANT, 448, 2> : norm_ring_kernel<XT, 2, QUANT, 512, 1>;
    return s.threads <= 256 ? norm_ring_kernel<XT, 1, QUANT, 256, 4> : norm_ring_kernel<XT, 1, QUANT, 512, 2>;
  };
  auto kern = f32 ? pick(static_cast<float *>(nullptr)) : pick(static_cast<__nv_bfloat16 *>(nullptr));
  const int smem = kRingHead + s.slots * slot.size;
  *st = allow_smem(reinterpret_cast<const void *>(kern), smem, dev.device);
  if (*st != NVFP4_OK) return true;
  const int64_t cap = static_cast<int64_t>(s.per_sm) * dev.sm_count;
  *st = check_launch(launch(kern, dim3(static_cast<unsigned>(a.m < cap ? a.m : cap)), dim3(s.threads), smem, stream, pdl, 1, a, ra), name);
  return true;
}

// Vectors a thread in the plain forward kernel, aligned rows: one while the rows are few (the call waits for one
// row's latency), two from four rows an SM on (fewer, wider threads: more bytes in flight per warp).  Many rows
// of up to 8192 channels go to the ring, so this decides for the one width that it does not hold (ring_slots).
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
  // (rows of single channels: one vector a thread where they fit, 1024 x 8191 63 -> 43 us)
  const Shape s = shape_of(n, vec ? forward_vpt(m, n, dev.sm_count) : 1);
  NormArgs a{x, ldx, (const __nv_bfloat16 *)y, ldy, (const __nv_bfloat16 *)w_post, (const __nv_bfloat16 *)w_pre,
             (const __nv_bfloat16 *)gate, ldg, residual_scale, eps, weight_offset, x_out, ldxo, (__nv_bfloat16 *)h, ldh,
             nullptr, nullptr, nullptr, m, static_cast<int>(n), 0};
  const bool f32 = x_type == NVFP4_DTYPE_F32;
  if (vec && forward_ring<false>(a, f32, (flags & NVFP4_FLAG_PDL) != 0, (cudaStream_t)stream, dev, flags, &st, "block_norm")) return st;
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
  if (forward_ring<true>(a, x_type == NVFP4_DTYPE_F32, (flags & NVFP4_FLAG_PDL) != 0, (cudaStream_t)stream, dev, flags, &st,
                         name))
    return st;
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
  // (the most teams of either kernel on any GPU this library runs on; sized without a device)
  const Shape s = shape_of(n, 1);
  int64_t teams = grad_teams(m, s, 160);
  if (!s.warp && teams < m) {
    const int64_t ring = 160LL * 4;
    teams = ring > teams ? (ring < m ? ring : m) : teams;
  }
  return static_cast<size_t>(teams) * 3 * static_cast<size_t>(n) * 4;
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
  if (flags & ~(uint32_t)(NVFP4_FLAG_PDL | NVFP4_FLAG_DEBUG_TIMEOUT)) return fail(NVFP4_ERR_INVALID_ARG, "%s: unknown flags 0x%x", name, flags);
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
  const int sms = dev.sm_count < 160 ? dev.sm_count : 160;
  const int bytes[5] = {static_cast<int>(n) * xe, dh ? static_cast<int>(n) * 2 : 0, dx_out ? static_cast<int>(n) * xe : 0,
                        y ? static_cast<int>(n) * 2 : 0, token_gate ? static_cast<int>(n) * 2 : 0};
  const Slot slot = slot_of(bytes);
  const RingShape rs = vec ? backward_ring_shape(m, n, slot.size, sms) : RingShape{};
  const int64_t ring_teams = static_cast<int64_t>(rs.per_sm) * sms;
  const int teams = rs.use ? static_cast<int>(m < ring_teams ? m : ring_teams) : grad_teams(m, s, sms);
  NormGradArgs a{(const __nv_bfloat16 *)dh, lddh, dx_out, lddxo, x_out, ldxo, (const __nv_bfloat16 *)y, ldy,
                 (const __nv_bfloat16 *)w_post, (const __nv_bfloat16 *)w_pre, (const __nv_bfloat16 *)gate, ldg,
                 residual_scale, eps, weight_offset, dx, lddx, (__nv_bfloat16 *)dy, lddy,
                 token_gate ? (__nv_bfloat16 *)dgate : nullptr, lddg, static_cast<float *>(workspace), m,
                 static_cast<int>(n), planes, teams};
  const bool pdl = (flags & NVFP4_FLAG_PDL) != 0, f32 = x_type == NVFP4_DTYPE_F32;
  cudaError_t e = cudaSuccess;
  if (rs.use) {
    const RingArgs ra{rs.slots, slot, dev.status, wait_limit(flags)};
    auto pick = [&](auto *x) {
      using XT = std::remove_pointer_t<decltype(x)>;
      if (rs.vpt == 2) return norm_grad_ring_kernel<XT, 2, 512, 1>;
      return rs.threads <= 128 ? norm_grad_ring_kernel<XT, 1, 128, 4>
                               : (rs.threads <= 256 ? norm_grad_ring_kernel<XT, 1, 256, 2> : norm_grad_ring_kernel<XT, 1, 512, 1>);
    };
    auto kern = f32 ? pick(static_cast<float *>(nullptr)) : pick(static_cast<__nv_bfloat16 *>(nullptr));
    const int smem = kRingHead + rs.slots * slot.size;
    st = allow_smem(reinterpret_cast<const void *>(kern), smem, dev.device);
    if (st != NVFP4_OK) return st;
    e = launch(kern, dim3(static_cast<unsigned>(teams)), dim3(rs.threads), smem, (cudaStream_t)stream, pdl, 1, a, ra);
  } else if (m > 0) {
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
    // (behind the kernel above with PDL whatever the flags: it waits for that kernel itself)
    e = launch(norm_colsum_kernel, dim3(static_cast<unsigned>(ceil_div(static_cast<int64_t>(planes) * n, 32))), dim3(32, 32), 0,
               (cudaStream_t)stream, pdl || m > 0, 1, (const float *)workspace, teams, planes, static_cast<int>(n), out[0], out[1], out[2]);
  }
  return check_launch(e, name);
}
