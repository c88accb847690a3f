// e4m3 quantisation with one fp32 scale per block of 128, along the rows, along the columns (transposed), both
// from one read, or per 128 x 128 block.
//
// A block with largest magnitude amax (at least 2^-100) has scale s = fl(amax / 448) and codes
// e4m3(fl(x * fl(448 / amax))): every step is one fp32 rounding to nearest even, so the codes are the same
// wherever a block is quantised.  A NaN outweighs every magnitude: a block that holds one, or an infinity, gets a
// scale and codes that stand for nothing finite.
//
// The least that any of it does is to move each value once in (2 or 4 bytes) and once or twice out (1 byte each).
// Along the rows and per 128 x 128 block memory bounds it: 8192 x 7168 bf16 28 us (6.3 TB/s), fp32 4096 x 7168 24 us
// (6.2); an fp32 weight of 4096 x 7168 and its transpose 29 us (6.0).  Both ways from one read is half bound by
// instructions (two products, two conversions and the exchange of the columns' magnitudes a value): 4096 x 7168 bf16
// 22 us (5.3 TB/s), and 32,768 rows of 2048 gathered from 4096, whose reads stay in L2, 47 us where the writes alone
// need 23.  Along the columns alone: 4096 x 7168 bf16 16 us (5.6 TB/s), fp32 27 (5.6).
#include "host.h"
#include "ptx.cuh"

namespace nvfp4 {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kMaxQuantExperts = 1024;
constexpr uint32_t kTinyBits = 27u << 23;  // 2^-100

// The larger magnitude, NaN above all; the sign of the result means nothing.  fp32, or two bf16 to a word.
template <bool F32>
__device__ __forceinline__ uint32_t mag_max(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (F32) {
    float f;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(f) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
    r = __float_as_uint(f);
  } else {
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  }
  return r;
}
__device__ __forceinline__ uint64_t both(float f) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(f));
  return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void split(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

// Sixteen consecutive values of a row, as loaded.
template <bool F32>
struct Vals {
  uint32_t w[F32 ? 16 : 8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (F32 ? 16 : 8); ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const void *p) {
    uint32_t a[8];
    ld_global_nc_v8(p, a);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = a[i];
    if constexpr (F32) {
      ld_global_nc_v8(static_cast<const uint8_t *>(p) + 32, a);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[8 + i] = a[i];
    }
  }
  // 16-byte loads, for rows that are not 32-byte aligned
  __device__ __forceinline__ void load16(const void *p) {
    const uint4 *q = static_cast<const uint4 *>(p);
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); ++i) {
      const uint4 v = __ldg(q + i);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  }
  // the bits of the largest magnitude, as fp32
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = w[0];
#pragma unroll
    for (int i = 1; i < (F32 ? 16 : 8); ++i) m = mag_max<F32>(m, w[i]);
    if constexpr (F32) return m & 0x7FFFFFFFu;
    return mag_max<true>(m & 0xFFFF0000u, m << 16) & 0x7FFFFFFFu;
  }
  // values 2 i and 2 i + 1, as a pair
  __device__ __forceinline__ uint64_t pair(int i) const {
    uint64_t r;
    if constexpr (F32) asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(w[2 * i]), "r"(w[2 * i + 1]));
    else asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(w[i] << 16), "r"(w[i] & 0xFFFF0000u));
    return r;
  }
};

__device__ __forceinline__ void divided(uint32_t amax_bits, float &scale, float &factor) {
  const float a = __uint_as_float(max(amax_bits, kTinyBits));
  scale = __fdiv_rn(a, 448.0f);
  factor = __fdiv_rn(448.0f, a);
}

// Four fp32 -> four e4m3 codes (RNE, saturating; NaN stays NaN), in byte order.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n"
      " cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
      " cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      " mov.b32 %0, {lo, hi};\n}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// The codes of a row's sixteen values under factor f.
template <bool F32>
__device__ __forceinline__ uint4 codes16(const Vals<F32> &v, float f) {
  const uint64_t f2 = both(f);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y[4];
    split(mul_pair(v.pair(2 * i), f2), y[0], y[1]);
    split(mul_pair(v.pair(2 * i + 1), f2), y[2], y[3]);
    o[i] = e4m3x4(y[0], y[1], y[2], y[3]);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// ------------------------------------------------------------------ along the rows only
// Eight lanes share a block of 128 (16 values each), a warp takes the same block of four rows, a CTA 32 rows
// and U blocks, whose loads are all in flight before the first is used.
template <bool F32, int U>
__global__ void __launch_bounds__(kQuantThreads) fp8_rows_kernel(const void *__restrict__ x, int64_t ldx,
                                                                 const int32_t *__restrict__ src, int64_t x_rows, int64_t m,
                                                                 int k, int kb, uint8_t *__restrict__ q,
                                                                 float *__restrict__ sf, int wide, unsigned int *status) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x % 32, cg = lane & 7;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32) * 4 + (lane >> 3);
  const int b0 = blockIdx.y * U;
  bool in = row < m;
  int64_t xr = in ? row : 0;
  if (src && in) {
    xr = src[row];
    if (xr < 0 || xr >= x_rows) {
      if (b0 == 0 && cg == 0) atomicOr(status, 8u);
      xr = -1;  // quantises zeros
    }
  }
  const uint8_t *xp = static_cast<const uint8_t *>(x) + (xr < 0 ? 0 : xr) * ldx * (F32 ? 4 : 2);
  Vals<F32> v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (b0 + u) * 128 + cg * 16;
    v[u].zero();
    if (in && xr >= 0 && c < k) {
      if (wide) v[u].load(xp + static_cast<int64_t>(c) * (F32 ? 4 : 2));
      else v[u].load16(xp + static_cast<int64_t>(c) * (F32 ? 4 : 2));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (b0 + u >= kb) break;
    uint32_t am = v[u].amax();
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
    float s, f;
    divided(am, s, f);
    const int c = (b0 + u) * 128 + cg * 16;
    if (in && c < k) *reinterpret_cast<uint4 *>(q + row * k + c) = codes16<F32>(v[u], f);
    if (in && cg == 0) sf[static_cast<int64_t>(b0 + u) * m + row] = s;
  }
}

// ------------------------------------------------------------------ 128 x 128 tiles
// What a tile is quantised along.
enum Along { kColumns = 0, kBoth = 1, kBlock = 2 };

struct TileArgs {
  const void *x;
  int64_t ldx, x_rows, m;      // m: rows of the result
  const int32_t *src;
  int k, kb;
  const int64_t *row_offsets;  // experts' rows (each expert's columns of qt begin at a multiple of 128)
  int experts;
  int64_t row_blocks;          // 128-row blocks of qt (kBlock: of one matrix)
  uint8_t *q;
  float *sf;
  uint8_t *qt;
  float *sft;
  int wide, chain;             // chain: consecutive tiles along k that a CTA takes
  unsigned int *status;
};

// One thread's part of a lane-transposed maximum: N values in each of the lanes that differ in the bits lo .. 2 lo ..
// (log2 N of them) come back as one value a lane, the maximum over those lanes of value
// (lane / lo) mod N with its bits reversed; an exchange halves the values that a lane still holds.
template <bool F32, int N>
__device__ __forceinline__ void exchange_max(uint32_t (&v)[N], int keep, int mask, int lane) {
  const bool up = (lane & mask) != 0;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    if (i < keep) {
      const uint32_t send = up ? v[i] : v[i + keep], mine = up ? v[i + keep] : v[i];
      v[i] = mag_max<F32>(mine, __shfl_xor_sync(0xFFFFFFFFu, send, mask));
    }
  }
}

// A warp holds 16 rows of the tile, a thread 4 rows x 16 columns (lane: column group cg = lane mod 8, row group
// rg = lane / 8).  The codes along the columns go through shared memory, four rows of a column to a word; the
// word's place is turned by its column group, so that the 32 lanes' words fall into 32 banks, and a column's 128
// bytes leave as eight 16-byte stores side by side.  A division for a row's scale or factor is done by one of the
// eight lanes that share the row.
template <bool F32, int ALONG>
__global__ void __launch_bounds__(kQuantThreads, F32 ? 2 : 3) fp8_tile_kernel(const TileArgs a) {
  constexpr int NW = F32 ? 16 : 8;  // words of a thread's 16 columns
  __shared__ uint32_t s_max[8][8 * NW];
  __shared__ __align__(16) float s_fac[128];
  __shared__ __align__(16) uint32_t s_t[2][128 * 32];
  __shared__ int s_scan[8];
  __shared__ int s_row0, s_rows;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, cg = lane & 7, rg = lane >> 3;
  const int64_t blk = blockIdx.x;
  int64_t row0, rows;           // first row of the result in this tile, rows in it
  int64_t mat = 0, mblk = blk;  // kBlock: matrix and its row block
  if (ALONG == kBlock) {
    mat = blk / a.row_blocks;
    mblk = blk % a.row_blocks;
    row0 = mat * a.m + mblk * 128;
    rows = min(static_cast<int64_t>(128), a.m - mblk * 128);
  } else if (a.row_offsets) {
    // the expert whose padded rows hold this block: a running sum over the experts, 256 at a time
    if (tid == 0) s_rows = 0;
    int64_t first = 0;
    bool bad = false;
    for (int e0 = 0; e0 < a.experts; e0 += kQuantThreads) {
      const int e = e0 + tid;
      int64_t lo = 0, hi = 0;
      if (e < a.experts) {
        lo = a.row_offsets[e];
        hi = a.row_offsets[e + 1];
        bad = bad || lo < 0 || hi < lo || hi > a.m || (e == 0 && lo != 0);
      }
      const int nb = bad ? 0 : static_cast<int>((hi - lo + 127) / 128);
      int incl = nb;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += n;
      }
      if (lane == 31) s_scan[warp] = incl;
      __syncthreads();
      int before = 0, all = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const int n = s_scan[w];
        before += w < warp ? n : 0;
        all += n;
      }
      const int64_t mine = first + before + incl - nb;
      if (nb > 0 && blk >= mine && blk < mine + nb) {
        s_row0 = static_cast<int>(lo + (blk - mine) * 128);
        s_rows = static_cast<int>(min(static_cast<int64_t>(128), hi - lo - (blk - mine) * 128));
      }
      first += all;
      __syncthreads();
    }
    const bool any_bad = __syncthreads_or(bad);
    if (any_bad && tid == 0 && blk == 0 && blockIdx.y == 0) atomicOr(a.status, 2u);
    row0 = s_row0;
    rows = any_bad ? 0 : s_rows;  // 0: past the last expert (or malformed offsets): the block is written as zeros
    if (rows == 0) row0 = 0;
  } else {
    row0 = blk * 128;
    rows = min(static_cast<int64_t>(128), a.m - row0);
  }
  const int b0 = blockIdx.y * a.chain, b1 = min(a.kb, b0 + a.chain);
  const int64_t ldt = ALONG == kBlock ? a.m : a.row_blocks * 128;
  const int ch = tid % 8;  // 16-byte piece of a column's 128 rows
  if (ALONG != kBlock && rows == 0) {  // zeros and their scale (one block in six where 128 experts share 32,768 rows)
    const int64_t c1 = min(static_cast<int64_t>(a.k), static_cast<int64_t>(b1) * 128);
    for (int64_t c = static_cast<int64_t>(b0) * 128 + tid / 8; c < c1; c += kQuantThreads / 8)
      *reinterpret_cast<uint4 *>(a.qt + c * ldt + blk * 128 + ch * 16) = make_uint4(0u, 0u, 0u, 0u);
    const float s = __fdiv_rn(__uint_as_float(kTinyBits), 448.0f);
    for (int64_t c = static_cast<int64_t>(b0) * 128 + tid; c < c1; c += kQuantThreads) a.sft[blk * a.k + c] = s;
    return;
  }
  // this thread's four rows
  const int r0 = warp * 16 + rg * 4;
  const uint8_t *xp[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int64_t xr = r0 + i < rows ? row0 + r0 + i : -1;
    if (ALONG != kBlock && a.src && xr >= 0) {
      xr = a.src[xr];
      if (xr < 0 || xr >= a.x_rows) {
        if (blockIdx.y == 0 && cg == 0) atomicOr(a.status, 8u);
        xr = -1;
      }
    }
    xp[i] = xr < 0 ? nullptr : static_cast<const uint8_t *>(a.x) + (xr * a.ldx + cg * 16) * (F32 ? 4 : 2);
  }
  // where this thread's codes go in the first tile: its rows', and its piece of the columns' (a column in 32)
  uint8_t *qp = ALONG == kColumns ? nullptr : a.q + (row0 + r0) * a.k + b0 * 128 + cg * 16;
  uint8_t *tp = nullptr;
  if (ALONG != kBlock) tp = a.qt + (static_cast<int64_t>(b0) * 128 + tid / 8) * ldt + blk * 128 + ch * 16;
  else if (a.qt) tp = a.qt + (mat * a.k + static_cast<int64_t>(b0) * 128 + tid / 8) * ldt + mblk * 128 + ch * 16;
  const bool piece_in = ALONG != kBlock || mblk * 128 + ch * 16 < a.m;
  for (int b = b0; b < b1; ++b) {
    const int c0 = b * 128;
    const bool in_k = c0 + cg * 16 < a.k;
    Vals<F32> v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i].zero();
      if (xp[i] && in_k) {
        const uint8_t *p = xp[i] + static_cast<int64_t>(c0) * (F32 ? 4 : 2);
        if (a.wide) v[i].load(p);
        else v[i].load16(p);
      }
    }
    // The next tile's rows into L1 meanwhile, where an expert's rows are read (32,768 of 2048 gathered from 4096: 49.4 ->
    // 47.4 us, not gathered 55.6 -> 52.7).  Plain rows, more tiles at once, lost by it (4096 x 7168 22.4 -> 23.5 us).
    if (ALONG != kBlock && a.row_offsets && b + 1 < b1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (xp[i] && c0 + 128 + cg * 16 < a.k)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(xp[i] + static_cast<int64_t>(c0 + 128) * (F32 ? 4 : 2)));
    }
    float fb = 0.0f;  // kBlock: the tile's factor
    if constexpr (ALONG == kBlock) {
      uint32_t am = max(max(v[0].amax(), v[1].amax()), max(v[2].amax(), v[3].amax()));
      am = __reduce_max_sync(0xFFFFFFFFu, am);
      if (lane == 0) s_max[warp][b & 1] = am;
      __syncthreads();
      am = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) am = max(am, s_max[w][b & 1]);
      const float top = __uint_as_float(max(am, kTinyBits));
      fb = __fdiv_rn(448.0f, top);
      if (tid == 0) {
        const float s = __fdiv_rn(top, 448.0f);
        a.sf[(mat * a.row_blocks + mblk) * a.kb + b] = s;
        if (a.qt) a.sft[(mat * a.kb + b) * a.row_blocks + mblk] = s;
      }
    }
    float fr[4] = {fb, fb, fb, fb};  // the rows' factors
    if constexpr (ALONG == kBoth) {
      // largest magnitudes of the four rows over their eight lanes: lane cg ends with row 2 (cg bit 0) + (cg bit 1)
      uint32_t am[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) am[i] = v[i].amax();
      exchange_max<true>(am, 2, 1, lane);
      exchange_max<true>(am, 1, 2, lane);
      const uint32_t m = mag_max<true>(am[0], __shfl_xor_sync(0xFFFFFFFFu, am[0], 4)) & 0x7FFFFFFFu;
      const float top = __uint_as_float(max(m, kTinyBits));
      // lanes 0 to 3 of the eight divide for the scales, 4 to 7 for the factors
      const float d = __fdiv_rn((cg & 4) ? 448.0f : top, (cg & 4) ? top : 448.0f);
      const int row = 2 * (cg & 1) + ((cg >> 1) & 1);
      if (cg < 4 && r0 + row < rows) a.sf[static_cast<int64_t>(b) * a.m + row0 + r0 + row] = d;
#pragma unroll
      for (int i = 0; i < 4; ++i) fr[i] = __shfl_sync(0xFFFFFFFFu, d, (lane & 24) | 4 | (i >> 1) | ((i & 1) << 1));
    }
    const bool turned = ALONG != kBlock || a.qt != nullptr;
    if constexpr (ALONG != kBlock) {
      // largest magnitude of each column: over the thread's rows, the warp's four row groups, the warps
      uint32_t am[NW];
#pragma unroll
      for (int j = 0; j < NW; ++j)
        am[j] = mag_max<F32>(mag_max<F32>(v[0].w[j], v[1].w[j]), mag_max<F32>(v[2].w[j], v[3].w[j]));
      exchange_max<F32>(am, NW / 2, 8, lane);
      exchange_max<F32>(am, NW / 4, 16, lane);
      // rg bit 0 chose the upper half of the words, bit 1 the upper half of that
#pragma unroll
      for (int j = 0; j < NW / 4; ++j) s_max[warp][cg * NW + (rg & 1) * (NW / 2) + (rg >> 1) * (NW / 4) + j] = am[j];
      __syncthreads();
      if (tid < 128) {
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = mag_max<F32>(m, s_max[w][F32 ? tid : tid / 2]);
        if constexpr (!F32) m = (tid & 1) ? (m & 0xFFFF0000u) : (m << 16);
        float s, fc;
        divided(m & 0x7FFFFFFFu, s, fc);
        s_fac[(tid & 12) * 8 + (tid >> 4) * 4 + (tid & 3)] = fc;  // the eight column groups' fours side by side
        if (c0 + tid < a.k) a.sft[blk * a.k + c0 + tid] = s;
      }
      __syncthreads();
    }
    // four columns at a time: their part of the rows' codes, and the four rows of each column's
    uint32_t *turn = s_t[b & 1];
    uint32_t o[4][4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint64_t x[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i][0] = v[i].pair(2 * g);
        x[i][1] = v[i].pair(2 * g + 1);
        if constexpr (ALONG != kColumns) {
          float y[4];
          split(mul_pair(x[i][0], both(fr[i])), y[0], y[1]);
          split(mul_pair(x[i][1], both(fr[i])), y[2], y[3]);
          o[i][g] = e4m3x4(y[0], y[1], y[2], y[3]);
        }
      }
      if (turned) {
        ulonglong2 f = make_ulonglong2(both(fb), both(fb));  // the columns' factors
        if constexpr (ALONG != kBlock) f = *reinterpret_cast<const ulonglong2 *>(&s_fac[g * 32 + cg * 4]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float lo[4], hi[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) split(mul_pair(x[i][j], j ? f.y : f.x), lo[i], hi[i]);
          const int c = cg * 16 + 4 * g + 2 * j;
          turn[c * 32 + ((warp * 4 + rg) ^ (cg * 4))] = e4m3x4(lo[0], lo[1], lo[2], lo[3]);
          turn[(c + 1) * 32 + ((warp * 4 + rg) ^ (cg * 4))] = e4m3x4(hi[0], hi[1], hi[2], hi[3]);
        }
      }
    }
    if constexpr (ALONG != kColumns) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r0 + i < rows && in_k)
          *reinterpret_cast<uint4 *>(qp + static_cast<int64_t>(i) * a.k) = make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
      qp += 128;
    }
    if (!turned) continue;
    __syncthreads();  // (the other of the two is written next, and this one again two tiles on, behind its barriers)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = i * 32 + tid / 8;
      if (c0 + c < a.k && piece_in)
        *reinterpret_cast<uint4 *>(tp + i * 32 * ldt) = *reinterpret_cast<const uint4 *>(&turn[c * 32 + ((ch * 4) ^ ((c / 16) * 4))]);
    }
    tp += 128 * ldt;
  }
}

nvfp4_status_t check_input(const char *name, const void *x, int x_type, int64_t ldx, int64_t k, int64_t rows) {
  if (x_type != NVFP4_DTYPE_BF16 && x_type != NVFP4_DTYPE_F32)
    return fail(NVFP4_ERR_INVALID_ARG, "%s: x_type=%d", name, x_type);
  if (rows < 0 || k <= 0 || rows > (1LL << 31) - 512 || k > (1LL << 31) - 512)
    return fail(NVFP4_ERR_INVALID_ARG, "%s: rows=%lld k=%lld", name, (long long)rows, (long long)k);
  if (k % 16) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: k=%lld is not a multiple of 16", name, (long long)k);
  const int unit = x_type == NVFP4_DTYPE_F32 ? 4 : 8;
  if ((ldx != 0 && ldx < k) || ldx % unit || !aligned(x, 16))
    return fail(NVFP4_ERR_MISALIGNED, "%s: x needs 16-B alignment and rows of at least k that start on 16 B (ldx=%lld)", name,
                (long long)ldx);
  return NVFP4_OK;
}
int wide_rows(const void *x, int x_type, int64_t ldx) {
  return aligned(x, 32) && ldx * (x_type == NVFP4_DTYPE_F32 ? 4 : 2) % 32 == 0;
}

template <int ALONG>
cudaError_t launch_tiles(int x_type, TileArgs &a, int64_t blocks, const DeviceInfo &dev, uint32_t flags, nvfp4_stream_t s) {
  // tiles that a CTA takes in turn, so that its rows' places are looked up once: at most 3, and no more than leave four
  // CTAs an SM (32,768 rows of 2048 over 128 experts, without the prefetch: 1 60 us, 2 52, 3 49, 4 50, 8 58)
  const int64_t tiles = blocks * a.kb, want = static_cast<int64_t>(dev.sm_count) * 4;
  int64_t chain = tiles / want;
  chain = chain < 1 ? 1 : chain > 3 ? 3 : chain;
  chain = ceil_div(a.kb, ceil_div(a.kb, chain));  // as many to every CTA
  a.chain = static_cast<int>(chain);
  auto kern = x_type == NVFP4_DTYPE_F32 ? fp8_tile_kernel<true, ALONG> : fp8_tile_kernel<false, ALONG>;
  return launch(kern, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(ceil_div(a.kb, chain))), dim3(kQuantThreads),
                0, (cudaStream_t)s, (flags & NVFP4_FLAG_PDL) != 0, 1, a);
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" int64_t fp8_padded_rows(int64_t rows, int num_experts) {
  if (rows < 0 || num_experts < 0) return 0;
  return round_up(rows, 128) + 128 * static_cast<int64_t>(num_experts);
}

extern "C" nvfp4_status_t fp8_quantize(const void *x, int x_type, int64_t x_rows, int64_t k, int64_t ldx,
                                       const int32_t *src_rows, int64_t rows, const int64_t *row_offsets, int num_experts,
                                       uint8_t *q, float *sf, uint8_t *qt, float *sft, uint32_t flags,
                                       nvfp4_stream_t stream) {
  clear_error();
  const char *name = "fp8_quantize";
  nvfp4_status_t st = check_input(name, x, x_type, ldx, k, rows);
  if (st != NVFP4_OK) return st;
  if (x_rows < 0 || (!src_rows && rows > 0 && rows != x_rows))
    return fail(NVFP4_ERR_INVALID_ARG, "%s: x_rows=%lld rows=%lld (equal without src_rows)", name, (long long)x_rows,
                (long long)rows);
  if (flags & ~(uint32_t)NVFP4_FLAG_PDL) return fail(NVFP4_ERR_INVALID_ARG, "%s: unknown flags 0x%x", name, flags);
  if ((q == nullptr) != (sf == nullptr) || (qt == nullptr) != (sft == nullptr) || (rows > 0 && !q && !qt))
    return fail(NVFP4_ERR_INVALID_ARG, "%s: q and sf, qt and sft: give both or neither, and one pair at least", name);
  if (row_offsets ? (num_experts < 1 || num_experts > kMaxQuantExperts) : num_experts != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "%s: num_experts=%d (1..%d with row_offsets, 0 without)", name, num_experts,
                kMaxQuantExperts);
  if (row_offsets && !qt) return fail(NVFP4_ERR_INVALID_ARG, "%s: row_offsets belong to qt", name);
  if (!aligned(q, 16) || !aligned(qt, 16) || !aligned(sf, 4) || !aligned(sft, 4) || !aligned(src_rows, 4) ||
      !aligned(row_offsets, 8))
    return fail(NVFP4_ERR_MISALIGNED, "%s: q and qt need 16-B, row_offsets 8-B, the others 4-B alignment", name);
  const int64_t blocks = fp8_padded_rows(rows, num_experts) / 128;
  if (blocks == 0 || (rows == 0 && !qt)) return NVFP4_OK;
  if (!x && rows > 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", name);
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  const int kb = static_cast<int>(ceil_div(k, 128)), wide = wide_rows(x, x_type, ldx);
  cudaError_t e;
  if (!qt) {
    // four blocks a CTA (their loads in flight together) once that still fills the device, one before
    const int64_t ctas = ceil_div(rows, 32);
    const int U = x_type == NVFP4_DTYPE_F32 ? 2 : 4;
    const bool many = ctas * ceil_div(kb, U) >= dev.sm_count * 4LL;
    if (ceil_div(kb, many ? U : 1) > 65535) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: k=%lld is too long", name, (long long)k);
    auto kern = x_type == NVFP4_DTYPE_F32 ? (many ? fp8_rows_kernel<true, 2> : fp8_rows_kernel<true, 1>)
                                          : (many ? fp8_rows_kernel<false, 4> : fp8_rows_kernel<false, 1>);
    e = launch(kern, dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(ceil_div(kb, many ? U : 1))), dim3(kQuantThreads), 0,
               (cudaStream_t)stream, (flags & NVFP4_FLAG_PDL) != 0, 1, x, ldx, src_rows, x_rows, rows, static_cast<int>(k), kb, q,
               sf, wide, dev.status);
    return check_launch(e, name);
  }
  if (kb > 65535) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: k=%lld is too long", name, (long long)k);
  TileArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.x_rows = x_rows;
  a.m = rows;
  a.src = src_rows;
  a.k = static_cast<int>(k);
  a.kb = kb;
  a.row_offsets = row_offsets;
  a.experts = num_experts;
  a.row_blocks = blocks;
  a.q = q;
  a.sf = sf;
  a.qt = qt;
  a.sft = sft;
  a.wide = wide;
  a.status = dev.status;
  e = q ? launch_tiles<kBoth>(x_type, a, blocks, dev, flags, stream) : launch_tiles<kColumns>(x_type, a, blocks, dev, flags, stream);
  return check_launch(e, name);
}

extern "C" nvfp4_status_t fp8_quantize_weight(const void *w, int w_type, int64_t matrices, int64_t n, int64_t k, int64_t ldw,
                                              uint8_t *q, float *sf, uint8_t *qt, float *sft, uint32_t flags,
                                              nvfp4_stream_t stream) {
  clear_error();
  const char *name = "fp8_quantize_weight";
  if (matrices < 0 || n < 0 || (n > 0 && matrices > ((1LL << 31) - 512) / n))
    return fail(NVFP4_ERR_INVALID_ARG, "%s: matrices=%lld n=%lld", name, (long long)matrices, (long long)n);
  nvfp4_status_t st = check_input(name, w, w_type, ldw, k, matrices * n);
  if (st != NVFP4_OK) return st;
  if (flags & ~(uint32_t)NVFP4_FLAG_PDL) return fail(NVFP4_ERR_INVALID_ARG, "%s: unknown flags 0x%x", name, flags);
  if ((qt == nullptr) != (sft == nullptr)) return fail(NVFP4_ERR_INVALID_ARG, "%s: qt and sft: give both or neither", name);
  if (qt && n % 16) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: the transpose needs n %% 16 == 0 (n=%lld)", name, (long long)n);
  if (!aligned(q, 16) || !aligned(qt, 16) || !aligned(sf, 4) || !aligned(sft, 4))
    return fail(NVFP4_ERR_MISALIGNED, "%s: q and qt need 16-B, the scales 4-B alignment", name);
  if (matrices == 0 || n == 0) return NVFP4_OK;
  if (!w || !q || !sf) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", name);
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  TileArgs a{};
  a.x = w;
  a.ldx = ldw;
  a.x_rows = a.m = n;
  a.k = static_cast<int>(k);
  a.kb = static_cast<int>(ceil_div(k, 128));
  if (a.kb > 65535) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: k=%lld is too long", name, (long long)k);
  a.row_blocks = ceil_div(n, 128);
  a.q = q;
  a.sf = sf;
  a.qt = qt;
  a.sft = sft;
  a.wide = wide_rows(w, w_type, ldw);
  a.status = dev.status;
  return check_launch(launch_tiles<kBlock>(w_type, a, matrices * a.row_blocks, dev, flags, stream), name);
}
