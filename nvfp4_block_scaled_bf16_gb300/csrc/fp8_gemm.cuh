// e4m3 products with one fp32 scale per block of 128 along K: D = sum over blocks b of
// (sP[row, b] sQ[col, b]) * sum over the block's 128 elements of P[row, k] Q[col, k].
//
// The tensor core sums one 128-wide block at a time into a tensor-memory buffer of its own (tcgen05.mma kind::f8f6f4,
// four instructions of K = 32), and scaling warps multiply that block's sums by its factor in fp32 and add them to
// accumulators that stay in registers over the whole K: the factor is an fp32 number, which no scale format of the
// tensor core holds.
//
// What bounds it, measured on 128 x 256 tiles (cycles a block).  The products alone take 512 (8192 multiply-adds a
// cycle), reading the sums 136 (0.53 a column and quarter of the SM).  Scaling with scalar multiply-adds slows the
// products to 930; with pairs (fma.rn.f32x2) they take 566 beside it, and the scaling 475, twice that with a factor per
// column too.  What is left of the 860 that a block takes (4096 x 4864 x 7168 in 106 us, 2.7 PFLOP/s; 1300 with a
// factor per column, 152 us) is the chain from a block's products through the scaling warps back to the buffer, and the
// test of the scales' range (see block_factors): without the loads of one operand it was 99 us where it was 103 with
// them.  Four warps to a scheduler hid more of it than two with more columns each (123 us then), than CTA pairs, which
// halve the operands' traffic but lengthen the chain (111 us), or than two CTAs an SM with 128 columns each (141 us).
//
// The operand whose rows lie in the 128 tensor-memory lanes is P, the other (the columns) is Q.
// Usually P is A (the tokens); with SWAP it is B (a weight), so that few tokens fill a narrow tile.
#pragma once

#include <cuda_bf16.h>

#include "host.h"
#include "ptx.cuh"

namespace nvfp4 {
namespace fp8 {

enum Mode { kDense = 0, kGrouped = 1, kWgrad = 2 };

constexpr int kMaxExperts = 1024;
constexpr int kGroup = 8;          // tiles along P that are taken in turn

template <int NT_, bool SWAP_, bool PV_, bool CV_, int MODE_>
struct Cfg {
  static constexpr int NT = NT_;         // columns of a tile (rows of Q)
  static constexpr bool SWAP = SWAP_;    // P is B
  static constexpr bool PV = PV_;        // P has a scale per row (else per 128 rows)
  static constexpr bool CV = CV_;        // Q has a scale per row
  static constexpr int MODE = MODE_;
  static constexpr int P_BYTES = 128 * 128;
  static constexpr int Q_BYTES = NT * 128;
  static constexpr int STAGE = P_BYTES + Q_BYTES;
  // Wide rows of D leave through shared memory as bulk copies, so that the scaling warps go on with the next tile.
  // (Stored directly, 32 rows at a time by 32 bytes each, a 128 x 256 tile took 3200 cycles.)
  static constexpr bool BULK = !SWAP && NT == 256;
  // Few tokens: two CTAs to an SM, so that the weight's split over CTAs leaves fewer SMs idle.
  static constexpr int CTAS = SWAP && NT <= 32 ? 2 : 1;
  static constexpr int STAGES_FIT = (BULK ? 147456 : 200 * 1024 / CTAS) / STAGE;
  static constexpr int STAGES = STAGES_FIT > 12 ? 12 : STAGES_FIT;
  // Ring of the blocks' scales, which are asked for LEAD blocks before they are announced.
  static constexpr int SLOTS = BULK ? 6 : 8, LEAD = BULK ? 2 : 4;
  static constexpr int NACC = NT >= 256 ? 2 : 4;
  static constexpr int TMEM = NACC * NT < 32 ? 32 : NACC * NT;
  static constexpr int SW = NT >= 256 ? 16 : 8;     // scaling warps (behind 4 that feed)
  static constexpr int THREADS = 128 + 32 * SW;
  static constexpr int W = NT * 4 / SW;  // columns of one scaling warp
  static constexpr int CH = W <= 32 ? W / 2 : NT >= 256 ? 16 : 32;  // columns loaded at a time
  static constexpr int SC_P = PV ? 128 : 4;
  static constexpr int SC_Q = CV ? NT : 4;
  static constexpr int SC_BYTES = (SC_P + SC_Q + (CV ? 4 : 0)) * 4;  // CV: and whether a column's scale is far out
  static constexpr int TABLE = MODE == kDense ? 0 : 2 * (kMaxExperts + 4) * 4;
  static constexpr int OUT = BULK ? 65536 : 0;  // 128 rows x 512 bytes
  // where rows of D that are not aligned are turned around (BULK: in OUT)
  static constexpr int TURN = SWAP || BULK ? 0 : SW * 32 * 9 * 4;
  static constexpr int CTRL = 512;
  static_assert(NACC <= STAGES, "a buffer's next block must have a stage of its own");
  static constexpr int SMEM = 1024 + STAGES * STAGE + OUT + SLOTS * SC_BYTES + TABLE + TURN + CTRL;
  // f8f6f4: fp32 sums (1 at bit 4), e4m3 operands (0 at bits 7 and 10), both K-major
  static constexpr uint32_t IDESC = (1u << 4) | (static_cast<uint32_t>(NT >> 3) << 17) |
                                    (static_cast<uint32_t>(128 >> 4) << 24);
  static_assert(CTAS * (SMEM + 1024) <= 233472, "smem");
};

// Where an operand's scales lie: of row r (or of its block of 128) and block b along K at
// p + expert * es + r * rs + b * ks (rs = 1 where each row has one).
struct Scales {
  const float *p;
  int64_t es, rs, ks;
};

// Division by a number that the host knows, for dividends below 2^31: the multiplication by a rounded-up reciprocal
// of Granlund and Montgomery (a tile's place takes two divisions, and every warp asks for it).
struct Divisor {
  uint32_t d, mul, shift;
  __host__ static Divisor of(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    return Divisor{d, static_cast<uint32_t>(((1ull << 32) * ((1ull << l) - d)) / d + 1), l};
  }
  __device__ __forceinline__ int quotient(int n) const {
    const uint32_t u = static_cast<uint32_t>(n);
    return static_cast<int>((__umulhi(mul, u) + u) >> shift);
  }
};

struct Args {
  Scales sp, sq;
  void *d;
  int64_t ldd, d_expert;     // elements
  int p_rows, q_rows;        // dense and wgrad: rows of P and Q; grouped: rows of the weight in both
  int nk;                    // blocks along K (dense and grouped)
  int p_tiles, q_tiles;      // tiles along the static operands
  Divisor per_expert, group; // p_tiles * q_tiles; kGroup * q_tiles
  Divisor tail;              // tiles along P of the last, shorter group
  int splits;                // dense with SWAP: CTAs of a cluster that share a tile's K
  int out_f32, accumulate;
  int bulk;                  // rows of D start on 16 bytes and are not accumulated: bulk copies
  const int64_t *row_offsets;
  int experts;
  int64_t total_rows;        // grouped: rows of A
  unsigned int *status;
  long long wait_limit;
  int skip_first_load;
};

struct Tile {
  int p0, q0, p_end, q_end;  // rows of P and Q that the tile covers, and where they end
  int py, qy;                // their first rows in the tensor maps
  int kb0, nk;               // first block along K and how many
  int expert;
};

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t pdesc, uint64_t qdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(pdesc), "l"(qdesc), "r"(idesc), "r"(accumulate));
}

// Lane 0's arrival, without a branch.
__device__ __forceinline__ void arrive_lane0(uint32_t bar, int lane) {
  asm volatile("{\n .reg .pred p;\n setp.eq.s32 p, %1, 0;\n @p mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(bar), "r"(lane)
               : "memory");
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// N consecutive tensor-memory columns of the warp's 32 lanes.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 32) {
    tmem_ld_32x32b_x32(taddr, r);
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
  } else {
    static_assert(N == 8, "columns");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  }
}
// Multiplies COLS consecutive tensor-memory columns of the warp's 32 lanes, each lane's by its own factor.
template <int COLS>
__device__ __forceinline__ void tmem_scale(uint32_t taddr, float factor) {
#pragma unroll
  for (int c = 0; c < COLS; c += 8) {
    uint32_t v[8];
    tmem_ld<8>(taddr + c, v);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(__fmul_rn(__uint_as_float(v[j]), factor));
    tmem_st_32x32b<8>(taddr + c, v);
  }
  tmem_st_wait();
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack2u(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2f(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// 4-byte global -> shared copy; zero where `ok` is false (the address is not read then).
__device__ __forceinline__ void cp_async_4(uint32_t dst, const float *src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The factor f of a block's sums v in this lane: the scale of its row, and with !CV that of the warp's columns too (with
// CV each column's comes from the table, v * column's scale * f).  The quantiser's scales lie in [2^-109, 2^120) and a
// nonzero v in [2^-18, 2^24.7), so that v times one of them, or their product, may leave fp32 where v times both does not.
// Where some lane's could (true is returned), the sums are multiplied by `first` and what is left is f:
//   !CV: where the two scales' product is no normal number (but for a row's scale of zero: a row past the end) `first` is
//        the lesser scale, f the greater;
//   CV:  where a column's scale of more than 2^103 lets v * scale overflow too early (the warp that loads the scales
//        says so behind them) `first` is the power of two in a row's scale below 1, f the rest of it, so that no result
//        changes but those that overflowed.
// The test costs the grouped products 5 to 9 % (32768 rows over 128 experts 124 -> 130 us, over 8 of 2048 x 1536 98 -> 106),
// 256-column tiles with a scale per column up to 5 % (4096 x 4864 x 7168: 146 -> 152), the others 1 to 3 %.  Anything in the
// loop over the columns costs more (4096 x 4096 x 7168, 104 us without, 105 with the test: a branch there 115, a second
// product 146).
template <class C>
__device__ __forceinline__ bool block_factors(const float *sc, int quad, int half, int lane, float &f, float &first) {
  const float sp = C::PV ? sc[quad * 32 + lane] : sc[0];
  first = 1.0f;
  if constexpr (C::CV) {
    f = sp;
    if (sc[C::SC_P + C::SC_Q] == 0.0f) return false;
    const uint32_t bits = __float_as_uint(sp);
    if (bits - 0x00800000u < 0x3F000000u) {  // a normal number below 1
      first = __uint_as_float(bits & 0x7F800000u);
      f = __uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u);
    }
  } else {
    const float sq = sc[C::SC_P + half * C::W / 128];
    f = sp * sq;
    const bool far = __float_as_uint(f) - 0x00800000u >= 0x7F000000u && sp != 0.0f;
    if (!__any_sync(0xFFFFFFFFu, far)) return false;
    if (far) {  // (selects, not fminf: a NaN stays)
      first = sp < sq ? sp : sq;
      f = sp < sq ? sq : sp;
    }
  }
  return true;
}
// Adds CH columns of a block's sums, times their factors, to the accumulators; cols: the columns' scales.
template <class C>
__device__ __forceinline__ void add_scaled(const uint32_t (&v)[C::CH], const float *cols, float f, uint64_t *sum) {
  const uint64_t f2 = pack2(f, f);
  if constexpr (C::CV) {
    const ulonglong2 *cs = reinterpret_cast<const ulonglong2 *>(cols);
#pragma unroll
    for (int j = 0; j < C::CH; j += 4) {
      const ulonglong2 s = cs[j / 4];
      sum[j / 2] = fma2(mul2f(pack2u(v[j], v[j + 1]), s.x), f2, sum[j / 2]);
      sum[j / 2 + 1] = fma2(mul2f(pack2u(v[j + 2], v[j + 3]), s.y), f2, sum[j / 2 + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < C::CH; j += 2) sum[j / 2] = fma2(pack2u(v[j], v[j + 1]), f2, sum[j / 2]);
  }
}

enum Site { kSiteLoad = 0, kSiteMmaStage = 2, kSiteScaleSlot = 4, kSiteScaleStage = 5, kSiteAcc = 6 };

// Tables of the grouped forms in shared memory: row offsets; first tile of each expert or (wgrad) its first
// block along K.
struct Tables {
  int *ro, *tp, *kb;
};

template <class C>
__device__ __forceinline__ int token_tile() {
  return C::SWAP ? C::NT : 128;
}

template <class C>
__device__ __forceinline__ Tile tile_at(const Args &a, const Tables &tb, int t) {
  Tile r;
  r.expert = 0;
  r.kb0 = 0;
  r.nk = a.nk;
  int pi, qi;
  if constexpr (C::MODE == kGrouped) {
    int lo = 0, hi = a.experts - 1;  // the last expert whose first tile is at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tb.tp[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    r.expert = lo;
    const int rows = tb.ro[lo + 1] - tb.ro[lo];
    const int tt = (rows + token_tile<C>() - 1) / token_tile<C>();
    const int l = t - tb.tp[lo];
    // an expert's token tiles are adjacent: CTAs that run at the same time share the weight's tile
    if constexpr (C::SWAP) {
      pi = l / tt;
      qi = l % tt;
      r.p0 = pi * 128;
      r.p_end = a.p_rows;
      r.py = lo * a.p_rows + r.p0;
      r.q0 = r.qy = tb.ro[lo] + qi * C::NT;
      r.q_end = tb.ro[lo + 1];
    } else {
      qi = l / tt;
      pi = l % tt;
      r.p0 = r.py = tb.ro[lo] + pi * 128;
      r.p_end = tb.ro[lo + 1];
      r.q0 = qi * C::NT;
      r.q_end = a.q_rows;
      r.qy = lo * a.q_rows + r.q0;
    }
    return r;
  }
  if constexpr (C::MODE == kWgrad) {
    r.expert = a.per_expert.quotient(t);
    t -= r.expert * static_cast<int>(a.per_expert.d);
    r.kb0 = tb.kb[r.expert];
    r.nk = tb.kb[r.expert + 1] - r.kb0;
  }
  // groups of tiles along P: what runs at the same time shares both operands through L2
  const int g = a.group.quotient(t), l = t - g * static_cast<int>(a.group.d);
  const int gs = min(kGroup, a.p_tiles - g * kGroup);
  qi = gs == kGroup ? l / kGroup : a.tail.quotient(l);
  pi = g * kGroup + l - qi * gs;
  r.p0 = r.py = pi * 128;
  r.q0 = r.qy = qi * C::NT;
  r.p_end = a.p_rows;
  r.q_end = a.q_rows;
  return r;
}

// Bulk stores of this thread: their sources have been read; they are complete.
__device__ __forceinline__ void bulk_store_read(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}
__device__ __forceinline__ void bulk_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// A warp's 32 rows of W columns through `stage` (64 columns of bf16 or 32 of fp32 to 4 KB) as boxes of 32 rows x 128
// bytes; a row's sixteen-byte pieces are turned by its number modulo 8 (the copies' 128-byte swizzle), which spreads
// 8 rows over all banks.  Rows and columns past D's ends (`end` columns) are left out by the copies, boxes that begin
// past them are not sent.
template <int W>
__device__ __forceinline__ void store_bulk(const CUtensorMap &map, int f32, int col, int end, int row, int expert, uint32_t stage, int lane,
                                           const uint64_t (&acc)[W / 2]) {
  constexpr int BOXES = W / 64;  // of bf16; fp32 takes two rounds
  const uint32_t mine = stage + lane * 128, turn = (lane & 7) * 16;
  bulk_store_read(lane);
  if (!f32) {
#pragma unroll
    for (int c = 0; c < 8 * BOXES; ++c) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack2(acc[c * 4 + i], lo, hi);
        w[i] = pack_bf16x2(lo, hi);
      }
      sts128(mine + (c / 8) * 4096 + (((c % 8) * 16) ^ turn), w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < BOXES; ++i)
        if (col + i * 64 < end) tma_store_3d(&map, stage + i * 4096, (col + i * 64) * 2, row, expert);
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h) bulk_store_read(lane);
#pragma unroll
    for (int c = 0; c < 8 * BOXES; ++c) {
      const uint64_t v0 = acc[h * W / 4 + c * 2], v1 = acc[h * W / 4 + c * 2 + 1];
      sts128(mine + (c / 8) * 4096 + (((c % 8) * 16) ^ turn), static_cast<uint32_t>(v0), static_cast<uint32_t>(v0 >> 32),
             static_cast<uint32_t>(v1), static_cast<uint32_t>(v1 >> 32));
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < BOXES; ++i)
        if (col + h * W / 2 + i * 32 < end) tma_store_3d(&map, stage + i * 4096, (col + h * W / 2 + i * 32) * 4, row, expert);
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
}

__device__ __forceinline__ void store_one(const Args &a, int64_t at, float v) {
  if (a.out_f32) {
    float *d = static_cast<float *>(a.d) + at;
    *d = a.accumulate ? *d + v : v;
  } else {
    static_cast<__nv_bfloat16 *>(a.d)[at] = __float2bfloat16_rn(v);
  }
}

// A warp's 32 rows (one a lane) of W columns to D, the lane's row at element `at`, `n` columns and the row `in`
// it.  Where every row of D starts on 16 bytes a lane writes its own row, 32 bytes at a time if it can (whole
// sectors); else 8 columns at a time are turned around through shared memory, so that 8 lanes write one row's
// neighbours (one by one, a warp's store would touch 32 sectors for 4 bytes each).
template <int W>
__device__ __forceinline__ void store_rows(const Args &a, int64_t at, int n, bool in, float *turn, int lane,
                                           const uint64_t (&acc)[W / 2]) {
  const int es = a.out_f32 ? 4 : 2;
  uint8_t *d = static_cast<uint8_t *>(a.d) + at * es;
  const bool vec = (a.ldd * es) % 16 == 0 && (a.d_expert * es) % 16 == 0;
  if (vec) {
    if (!in) return;
    const bool wide = (reinterpret_cast<uintptr_t>(d) & 31) == 0;
    if (a.out_f32) {
#pragma unroll
      for (int c = 0; c < W; c += 8) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack2(acc[c / 2 + i], v[2 * i], v[2 * i + 1]);
        float *o = reinterpret_cast<float *>(d) + c;
        if (a.accumulate) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < n) v[i] += o[i];
        }
        if (c + 8 <= n) {
          if (wide) {
            const uint32_t w[8] = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]),
                                   __float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
            st_global_v8(o, w);
          } else {
            reinterpret_cast<float4 *>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < n) o[i] = v[i];
        }
      }
      return;
    }
#pragma unroll
    for (int c = 0; c < W; c += (W < 16 ? W : 16)) {
      constexpr int N = W < 16 ? W : 16;
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        float lo, hi;
        unpack2(acc[c / 2 + i], lo, hi);
        w[i] = pack_bf16x2(lo, hi);
      }
      uint16_t *o = reinterpret_cast<uint16_t *>(d) + c;
      if (N == 16 && wide && c + 16 <= n) {
        st_global_v8(o, w);
      } else {
#pragma unroll
        for (int g = 0; g < N; g += 8) {
          if (c + g + 8 <= n) {
            *reinterpret_cast<uint4 *>(o + g) = make_uint4(w[g / 2], w[g / 2 + 1], w[g / 2 + 2], w[g / 2 + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c + g + i < n) o[g + i] = static_cast<uint16_t>(w[(g + i) / 2] >> (16 * (i & 1)));
          }
        }
      }
    }
    return;
  }
  const uint32_t rows = __ballot_sync(0xFFFFFFFFu, in);
  const int64_t at0 = __shfl_sync(0xFFFFFFFFu, at, 0);  // lane 0's row; the others follow at ldd
#pragma unroll
  for (int c = 0; c < W; c += 8) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float lo, hi;
      unpack2(acc[(c + i) / 2], lo, hi);
      turn[lane * 9 + i] = lo;
      turn[lane * 9 + i + 1] = hi;
    }
    __syncwarp();
    const int j = lane & 7;
    if (c + j < n) {
#pragma unroll 4
      for (int r = lane >> 3; r < 32; r += 4)
        if (rows >> r & 1) store_one(a, at0 + r * a.ldd + c + j, turn[r * 9 + j]);
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::CTAS)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                    const __grid_constant__ CUtensorMap map_d, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  // the ring begins on a 1024-byte boundary (the swizzle's period)
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t *out = smem + C::STAGES * C::STAGE;  // 1024-byte aligned too
  float *scales = reinterpret_cast<float *>(out + C::OUT);
  uint8_t *ctrl = reinterpret_cast<uint8_t *>(scales) + C::SLOTS * C::SC_BYTES;
  // A block's products wait for one barrier and announce one: `full` collects the operands, the scales and the
  // scaling warps that emptied the block's buffer (NACC blocks before); `done` tells the loader that the stage and
  // the scaling warps that the sums are theirs.  Every wait and every commit of the issuing thread costs about 90
  // cycles that the tensor core does not work through (measured; a block's products take 512).
  uint64_t *full = reinterpret_cast<uint64_t *>(ctrl);  // [STAGES]
  uint64_t *done = full + C::STAGES;                    // [STAGES]
  uint64_t *sempty = done + C::STAGES;                  // [C::SLOTS] the scaling warps have read the scales
  uint64_t *drain = sempty + C::SLOTS;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
  int *abort_flag = reinterpret_cast<int *>(tmem_holder + 1);
  int *issued_count = abort_flag + 1;
  int *bad = issued_count + 1;
  Tables tb;
  tb.ro = reinterpret_cast<int *>(ctrl + C::CTRL);
  tb.tp = tb.kb = tb.ro + kMaxExperts + 4;
  float *turn = reinterpret_cast<float *>(C::BULK ? out : ctrl + C::CTRL + C::TABLE);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr bool SPLIT = C::MODE == kDense && C::SWAP;
  const int splits = SPLIT ? a.splits : 1;
  const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / splits, units = gridDim.x / splits;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(smem_u32(&full[i]), 2 + C::SW);
      mbar_init(smem_u32(&done[i]), 1);
    }
    for (int i = 0; i < C::SLOTS; ++i) mbar_init(smem_u32(&sempty[i]), C::SW);
    mbar_init(smem_u32(drain), 1);
    fence_barrier_init();
    *abort_flag = 0;
    *issued_count = 0;
    *bad = 0;
    prefetch_tmap(&map_p);
    prefetch_tmap(&map_q);
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_u32(tmem_holder), C::TMEM);
    tmem_relinquish<1>();
  }
  pdl_trigger();
  pdl_wait();
  int total = 0;
  if constexpr (C::MODE != kDense) {
    __syncthreads();  // *bad is clear
    for (int e = threadIdx.x; e <= a.experts; e += C::THREADS) {
      const int64_t v = a.row_offsets[e];
      const int64_t prev = e > 0 ? a.row_offsets[e - 1] : 0;
      // (wgrad: total_rows is the number of padded rows that the operands hold)
      if (v < prev || v > a.total_rows || (e == 0 && v != 0)) *bad = 1;
      tb.ro[e] = static_cast<int>(v);
    }
    __syncthreads();
    if (warp == 0) {
      int tiles = 0, blocks = 0;
      for (int b = 0; b < a.experts; b += 32) {
        const int e = b + lane;
        const int rows = e < a.experts ? tb.ro[e + 1] - tb.ro[e] : 0;
        int nt = rows > 0 ? (rows + token_tile<C>() - 1) / token_tile<C>() * (C::SWAP ? a.p_tiles : a.q_tiles) : 0;
        int nb = rows > 0 ? (rows + 127) / 128 : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xFFFFFFFFu, nt, o), y = __shfl_up_sync(0xFFFFFFFFu, nb, o);
          if (lane >= o) {
            nt += x;
            nb += y;
          }
        }
        if (e < a.experts) {
          if (C::MODE == kGrouped) tb.tp[e + 1] = tiles + nt;
          else tb.kb[e + 1] = blocks + nb;
        }
        tiles += __shfl_sync(0xFFFFFFFFu, nt, 31);
        blocks += __shfl_sync(0xFFFFFFFFu, nb, 31);
      }
      if (lane == 0) {
        tb.tp[0] = tb.kb[0] = 0;
        if (C::MODE == kWgrad && static_cast<int64_t>(blocks) * 128 > a.total_rows) *bad = 1;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if constexpr (C::MODE == kDense) total = a.p_tiles * a.q_tiles;
  else if constexpr (C::MODE == kGrouped) total = tb.tp[a.experts];
  else total = a.experts * a.p_tiles * a.q_tiles;
  if (C::MODE != kDense && *bad) {
    if (threadIdx.x == 0) atomicOr(a.status, 2u);
    total = 0;
  }
  const uint32_t tmem = *tmem_holder;
  const WaitCtl wc{a.wait_limit, abort_flag, a.status};

  // this CTA's share of a tile's blocks along K
  auto k_range = [&](const Tile &t, int &k0, int &k1) {
    k0 = 0;
    k1 = t.nk;
    if constexpr (SPLIT) {
      k0 = static_cast<int>(static_cast<int64_t>(t.nk) * rank / splits);
      k1 = static_cast<int>(static_cast<int64_t>(t.nk) * (rank + 1) / splits);
    }
  };

  uint64_t acc[C::W / 2];  // pairs of columns
  if (warp < 4) {
    // (640 threads begin with 96 registers; 4 warps at 40 and 16 at 104 need 91 of them.  56 instead of 40 gives the
    // scaling warps no less, but the compiler spilled more there: 107 and 156 us where it was 103 and 145.)
    if constexpr (C::SW == 16) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      // ------------------------------------------------------------ operands
      if (lane == 0) {
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = unit; u < total && ok; u += units) {
          const Tile t = tile_at<C>(a, tb, u);
          int k0, k1;
          k_range(t, k0, k1);
          for (int kb = k0; kb < k1; ++kb) {
            if (issued >= C::STAGES && !mbar_wait(smem_u32(&done[stage]), phase ^ 1, wc, kSiteLoad)) {
              ok = false;
              break;
            }
            const uint32_t bar = smem_u32(&full[stage]);
            const uint32_t dst = smem_u32(smem + stage * C::STAGE);
            const int x = (t.kb0 + kb) * 128;
            mbar_arrive_expect_tx(bar, C::STAGE);
            if (!(a.skip_first_load && issued == 0)) {
              tma_load_2d(dst, &map_p, bar, x, t.py);
              tma_load_2d(dst + C::P_BYTES, &map_q, bar, x, t.qy);
            }
            ++issued;
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        *issued_count = issued;
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ products
      // The whole warp keeps the loop, so that descriptors stay in uniform registers; one lane issues.
      int stage = 0, ab = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint64_t desc0 = sdesc_k_sw128(smem_u32(smem));
      for (int u = unit; u < total && ok; u += units) {
        const Tile t = tile_at<C>(a, tb, u);
        int k0, k1;
        k_range(t, k0, k1);
        for (int kb = k0; kb < k1; ++kb) {
          ok = mbar_wait(smem_u32(&full[stage]), phase, wc, kSiteMmaStage);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint64_t pd = desc0 + static_cast<uint32_t>(stage * (C::STAGE >> 4));
          const uint64_t qd = pd + (C::P_BYTES >> 4);
          const uint32_t d = tmem + ab * C::NT;
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_f8(d, pd + 2 * i, qd + 2 * i, C::IDESC, i > 0 ? 1u : 0u);
            tc_commit(smem_u32(&done[stage]));
          }
          __syncwarp();
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1;
          }
          if (++ab == C::NACC) ab = 0;
        }
      }
    } else {
      // ------------------------------------------------------------ scales: warp 2 even blocks, warp 3 odd ones
      const int mine = warp - 2;
      int i = mine;    // this warp's next block
      int block = 0;   // the tiles' next block
      bool ok = true;
      // block i - SLOTS has been read
      auto slot_free = [&]() -> bool {
        const bool is = i < C::SLOTS || mbar_wait(smem_u32(&sempty[i % C::SLOTS]), (i / C::SLOTS - 1) & 1, wc, kSiteScaleSlot);
        return __all_sync(0xFFFFFFFFu, is);
      };
      // what was asked for block n = i - LEAD has landed: announce it, once the block that had its stage before is done
      auto announce = [&]() {
        cp_async_commit();
        const int n = i - C::LEAD;
        if (n >= 0) {
          cp_async_wait_group<C::LEAD / 2>();
          if (n >= C::STAGES) {
            const bool is = mbar_wait(smem_u32(&done[n % C::STAGES]), (n / C::STAGES - 1) & 1, wc, kSiteScaleStage);
            ok = __all_sync(0xFFFFFFFFu, is);
          }
          __syncwarp();
          if constexpr (C::CV) {  // see block_factors
            float *sc = scales + (n % C::SLOTS) * (C::SC_BYTES / 4);
            float most = sc[C::SC_P + (C::NT < 32 ? lane % C::NT : lane)];
#pragma unroll
            for (int j = 1; j < C::NT / 32; ++j) most = fmaxf(most, sc[C::SC_P + j * 32 + lane]);
            const bool far = __any_sync(0xFFFFFFFFu, most > 0x1p103f);
            if (lane == 0) sc[C::SC_P + C::SC_Q] = far ? 1.0f : 0.0f;
          }
          if (ok) arrive_lane0(smem_u32(&full[n % C::STAGES]), lane);
        }
        i += 2;
      };
      for (int u = unit; u < total && ok; u += units) {
        const Tile t = tile_at<C>(a, tb, u);
        int k0, k1;
        k_range(t, k0, k1);
        // where this lane's scales of the tile's rows lie (a scale per row: the rows' lie side by side)
        const int pr = C::PV ? t.p0 + lane : 0, qr = C::CV ? t.q0 + lane : min(t.q0 + lane * 128, t.q_end - 1);
        const float *pp = a.sp.p + t.expert * a.sp.es + (C::PV ? pr : t.p0 / 128 * a.sp.rs) + t.kb0 * a.sp.ks;
        const float *qp = a.sq.p + t.expert * a.sq.es + (C::CV ? qr : qr / 128 * a.sq.rs) + t.kb0 * a.sq.ks;
        for (int kb = k0; kb < k1 && ok; ++kb, ++block) {
          if ((block & 1) != mine) continue;
          ok = slot_free();
          if (!ok) break;
          const uint32_t dst = smem_u32(scales) + (i % C::SLOTS) * C::SC_BYTES + lane * 4;
          const float *pb = pp + kb * a.sp.ks, *qb = qp + kb * a.sq.ks;
          // (rows past the end get zeros, and nothing is read for them)
          if constexpr (C::PV) {
#pragma unroll
            for (int j = 0; j < 4; ++j) cp_async_4(dst + j * 128, pr + j * 32 < t.p_end ? pb + j * 32 : a.sp.p, pr + j * 32 < t.p_end);
          } else if (lane == 0) {
            cp_async_4(dst, pb, true);
          }
          if constexpr (C::CV) {
#pragma unroll
            for (int j = 0; j < (C::NT + 31) / 32; ++j)
              if (C::NT >= 32 || lane < C::NT)
                cp_async_4(dst + C::SC_P * 4 + j * 128, qr + j * 32 < t.q_end ? qb + j * 32 : a.sq.p, qr + j * 32 < t.q_end);
          } else if (lane < (C::NT + 127) / 128) {
            cp_async_4(dst + C::SC_P * 4, qb, true);
          }
          announce();
        }
      }
      const int end = block + C::LEAD;
      while (ok && i < end && block > 0) {  // the last blocks
        ok = slot_free();
        if (ok) announce();
      }
      cp_async_wait_all();
    }
  } else {
    // -------------------------------------------------------------- scaling and sums
    if constexpr (C::SW == 16) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * C::W;
    int slot = 0, ab = 0, stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = 0; i < C::NACC; ++i) arrive_lane0(smem_u32(&full[i]), lane);  // the first blocks' buffers are empty
    for (int u = unit; u < total && ok; u += units) {
      const Tile t = tile_at<C>(a, tb, u);
      int k0, k1;
      k_range(t, k0, k1);
#pragma unroll
      for (int i = 0; i < C::W / 2; ++i) acc[i] = 0;
      if constexpr (C::SW == 16) {
        // four warps to a scheduler: one's waits pass while the others have work
        for (int kb = k0; kb < k1; ++kb) {
          if constexpr (C::CV) {  // (three counters fewer in 104 registers: weight gradients 229 -> 221 us, but others lose)
            static_assert(C::SLOTS == 2 * C::STAGES && C::SLOTS % C::NACC == 0, "the slot gives a block's other places");
            phase = slot >= C::STAGES ? 1u : 0u;
            stage = slot >= C::STAGES ? slot - C::STAGES : slot;
            ab = slot % C::NACC;
          }
          const bool ready = mbar_try_wait(smem_u32(&done[stage]), phase);
          if (!__all_sync(0xFFFFFFFFu, ready)) ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&done[stage]), phase, wc, kSiteAcc));
          if (!ok) break;
          tc_fence_after();
          const float *sc = scales + slot * (C::SC_BYTES / 4);
          float f, first;
          if (block_factors<C>(sc, quad, half, lane, f, first)) tmem_scale<C::W>(t_lane + ab * C::NT, first);
#pragma unroll
          for (int c = 0; c < C::W; c += C::CH) {
            uint32_t v[C::CH];
            tmem_ld<C::CH>(t_lane + ab * C::NT + c, v);
            tmem_ld_wait();
            if (c + C::CH == C::W) {
              tc_fence_before();
              const int next = stage + C::NACC >= C::STAGES ? stage + C::NACC - C::STAGES : stage + C::NACC;
              arrive_lane0(smem_u32(&full[next]), lane);
            }
            add_scaled<C>(v, sc + C::SC_P + half * C::W + c, f, acc + c / 2);
          }
          __syncwarp();
          arrive_lane0(smem_u32(&sempty[slot]), lane);
          if (++slot == C::SLOTS) slot = 0;
          if constexpr (!C::CV) {
            if (++ab == C::NACC) ab = 0;
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
      } else {
        // The barrier of the next block is tested while the last columns but one are added, and its first columns are
        // loaded before the last are: what the test, the loads and the scale take passes while there is work.
        constexpr int CHUNKS = C::W / C::CH;
        static_assert(CHUNKS >= 2 && CHUNKS % 2 == 0, "chunks");
        uint32_t r[2][C::CH];
        const float *sc = scales;
        // starts on a block whose sums (and so its scales) are there
        auto begin = [&]() {
          tc_fence_after();
          tmem_ld<C::CH>(t_lane + ab * C::NT, r[0]);
          sc = scales + slot * (C::SC_BYTES / 4);
        };
        // the whole warp goes on or gives up
        auto wait_done = [&](bool ready) {
          if (!__all_sync(0xFFFFFFFFu, ready)) ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&done[stage]), phase, wc, kSiteAcc));
        };
        if (k0 < k1) {
          wait_done(false);
          if (ok) begin();
        }
        for (int kb = k0; kb < k1 && ok; ++kb) {
          const float *scb = sc;
          float f, first;
          if (block_factors<C>(sc, quad, half, lane, f, first)) {
            tmem_ld_wait();
            tmem_scale<C::W>(t_lane + ab * C::NT, first);
            tmem_ld<C::CH>(t_lane + ab * C::NT, r[0]);
          }
          const int slot_b = slot, ab_b = ab;
          const int next = stage + C::NACC >= C::STAGES ? stage + C::NACC - C::STAGES : stage + C::NACC;  // the buffer's next block's stage
          const bool more = kb + 1 < k1;
          bool ready = false;
          if (++slot == C::SLOTS) slot = 0;
          if (++ab == C::NACC) ab = 0;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1;
          }
#pragma unroll
          for (int i = 0; i < CHUNKS; ++i) {
            if (i + 1 == CHUNKS && more) wait_done(ready);
            tmem_ld_wait();
            if (i + 1 < CHUNKS) {
              tmem_ld<C::CH>(t_lane + ab_b * C::NT + (i + 1) * C::CH, r[(i + 1) & 1]);
              if (i + 2 == CHUNKS && more) ready = mbar_try_wait(smem_u32(&done[stage]), phase);
            } else {  // the last columns are in registers: the buffer may be overwritten
              tc_fence_before();
              arrive_lane0(smem_u32(&full[next]), lane);
              if (more && ok) begin();
            }
            add_scaled<C>(r[i & 1], scb + C::SC_P + half * C::W + i * C::CH, f, acc + i * C::CH / 2);
          }
          __syncwarp();
          arrive_lane0(smem_u32(&sempty[slot_b]), lane);
        }
      }
      if (!ok || splits > 1 || (a.accumulate && k0 == k1)) continue;
      const int p = t.p0 + quad * 32 + lane, q = t.q0 + half * C::W;
      if constexpr (C::SWAP) {
        if (p < t.p_end) {
          const int64_t at = t.expert * a.d_expert + static_cast<int64_t>(q) * a.ldd + p;
#pragma unroll
          for (int i = 0; i < C::W; ++i) {
            float lo, hi;
            unpack2(acc[i / 2], lo, hi);
            if (q + i < t.q_end) store_one(a, at + i * a.ldd, (i & 1) ? hi : lo);
          }
        }
      } else {
        if constexpr (C::BULK) {
          const int p32 = t.p0 + quad * 32;
          // (rows past an expert's last belong to the next one: only a warp whose rows are all inside, or end with D)
          if (a.bulk && (C::MODE != kGrouped || p32 + 32 <= t.p_end)) {
            if (p32 < t.p_end && q < t.q_end)
              store_bulk<C::W>(map_d, a.out_f32, q, t.q_end, p32, C::MODE == kWgrad ? t.expert : 0,
                               smem_u32(out) + (warp - 4) * (C::OUT / C::SW), lane, acc);
            continue;
          }
          bulk_store_read(lane);  // what is still being copied out of the place that is turned around in
        }
        store_rows<C::W>(a, t.expert * a.d_expert + static_cast<int64_t>(p) * a.ldd + q, t.q_end - q, p < t.p_end,
                         turn + (warp - 4) * (C::BULK ? C::OUT / 4 / C::SW : 32 * 9), lane, acc);
      }
    }
  }

  if constexpr (C::BULK) {
    if (warp >= 4 && lane == 0) bulk_store_done();
  }

  // -------------------------------------------------------------- end
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // wait (bounded) for copies still landing and for outstanding products, so that nothing writes
    // shared or tensor memory after the CTA is gone (the stages' barriers wait for other arrivals too, that may
    // never come: 2^25 cycles are ample for a copy)
    if (threadIdx.x == 0) {
      const int issued = *issued_count;
      for (int i = issued > C::STAGES ? issued - C::STAGES : 0; i < issued; ++i) {
        const uint32_t bar = smem_u32(&full[i % C::STAGES]);
        const long long t0 = clock64();
        while (!mbar_try_wait(bar, (i / C::STAGES) & 1) && clock64() - t0 < (1LL << 25)) {
        }
      }
    }
    if (threadIdx.x == 32) {
      tc_commit(smem_u32(drain));
      const long long t0 = clock64();
      while (!mbar_try_wait(smem_u32(drain), 0) && clock64() - t0 < a.wait_limit) {
      }
    }
    __syncthreads();
  }
  if constexpr (SPLIT) {
    if (splits > 1) {
      // Each CTA of the cluster holds the sums over its part of K; they are laid down in the (now idle)
      // ring, columns outermost, and each CTA adds a share of the columns in rank order.
      float *red = reinterpret_cast<float *>(smem);
      if (warp >= 4) {
        const int row = (warp & 3) * 32 + lane, half = (warp - 4) >> 2;
#pragma unroll
        for (int i = 0; i < C::W; ++i) {
          float lo, hi;
          unpack2(acc[i / 2], lo, hi);
          red[(half * C::W + i) * 128 + row] = (i & 1) ? hi : lo;
        }
      }
      cluster_sync();
      const Tile t = tile_at<C>(a, tb, unit);
      const int cols = min(C::NT, t.q_end - t.q0);
      // 32 float4 a column
      for (int i = threadIdx.x + rank * C::THREADS; i < cols * 32; i += C::THREADS * splits) {
        const uint32_t off = smem_u32(red) + i * 16;
        float4 part[8];  // every CTA's, asked for together
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < splits) part[r] = ld_cluster_v4(map_to_rank(off, r));
        float4 s = part[0];
#pragma unroll
        for (int r = 1; r < 8; ++r)
          if (r < splits) s = make_float4(s.x + part[r].x, s.y + part[r].y, s.z + part[r].z, s.w + part[r].w);
        const int p = t.p0 + (i % 32) * 4;
        const int64_t at = static_cast<int64_t>(t.q0 + i / 32) * a.ldd + p;
        const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (p + j < t.p_end) store_one(a, at + j, v[j]);
      }
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, C::TMEM);
  }
  if (splits > 1) cluster_sync();  // no CTA leaves while another reads its memory
}

// What the products' entry points check and fill alike.  rows, cols: of the result; k: what is summed over.
inline nvfp4_status_t check_product(const char *name, int64_t rows, int64_t cols, int64_t k, int d_type, int accumulate,
                                    uint32_t flags) {
  constexpr int64_t kMost = (1LL << 31) - 512;  // tile origins step past the ends by less
  if (rows < 0 || cols <= 0 || k <= 0 || rows > kMost || cols > kMost || k > kMost)
    return fail(NVFP4_ERR_INVALID_ARG, "%s: sizes %lld, %lld, %lld", name, (long long)rows, (long long)cols, (long long)k);
  if (k % 16) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: k=%lld is not a multiple of 16", name, (long long)k);
  if (d_type != NVFP4_DTYPE_BF16 && d_type != NVFP4_DTYPE_F32)
    return fail(NVFP4_ERR_INVALID_ARG, "%s: d_type=%d", name, d_type);
  if (accumulate && d_type != NVFP4_DTYPE_F32)
    return fail(NVFP4_ERR_INVALID_ARG, "%s: only an fp32 result is accumulated", name);
  if (flags & ~(uint32_t)(NVFP4_FLAG_PDL | NVFP4_FLAG_DEBUG_TIMEOUT | NVFP4_FLAG_DEBUG_SKIP_FIRST_LOAD))
    return fail(NVFP4_ERR_INVALID_ARG, "%s: unknown flags 0x%x", name, flags);
  return NVFP4_OK;
}
inline void fill_args(Args &a, void *d, int d_type, int accumulate, int64_t ldd, int64_t k, const DeviceInfo &dev,
                      uint32_t flags) {
  a.d = d;
  a.out_f32 = d_type == NVFP4_DTYPE_F32;
  a.accumulate = accumulate != 0;
  a.ldd = ldd;
  a.nk = static_cast<int>(ceil_div(k, 128));
  a.splits = 1;
  a.status = dev.status;
  a.wait_limit = wait_limit(flags);
  a.skip_first_load = (flags & NVFP4_FLAG_DEBUG_SKIP_FIRST_LOAD) && (flags & NVFP4_FLAG_DEBUG_TIMEOUT);
}

// Tensor maps, shared memory and launch of one configuration.  tiles: an upper bound of the tiles (the
// grid is the smaller of that and what the device holds at once).
template <class C>
nvfp4_status_t launch_gemm(const char *name, const uint8_t *p, int64_t p_rows, const uint8_t *q, int64_t q_rows,
                           int64_t k, int64_t tiles, const Args &given, const DeviceInfo &dev, uint32_t flags,
                           nvfp4_stream_t stream) {
  CUtensorMap mp, mq;
  nvfp4_status_t st = encode_tmap_2d_u8(&mp, p, k, p_rows, k, 128, 128, true);
  if (st == NVFP4_OK) st = encode_tmap_2d_u8(&mq, q, k, q_rows, k, 128, C::NT, true);
  if (st != NVFP4_OK) return st;
  // D [experts (1 but for the weight gradients), rows, ldd]
  Args args = given;
  if (C::MODE != kGrouped) {
    args.per_expert = Divisor::of(static_cast<uint32_t>(args.p_tiles) * args.q_tiles);  // (the tiles are fewer than 2^31)
    args.group = Divisor::of(static_cast<uint32_t>(kGroup) * args.q_tiles);
    args.tail = Divisor::of(static_cast<uint32_t>(args.p_tiles % kGroup ? args.p_tiles % kGroup : 1));
  }
  CUtensorMap md = mp;
  const int64_t es = args.out_f32 ? 4 : 2;
  // (a copy's place in a row is 32 signed bits of bytes)
  args.bulk = C::BULK && !args.accumulate && args.ldd * es % 16 == 0 && args.d_expert * es % 16 == 0 && args.ldd * es < (1LL << 31);
  if (args.bulk) {
    const int64_t rows = C::MODE == kWgrad ? args.p_rows : p_rows, depth = C::MODE == kWgrad ? args.experts : 1;
    st = encode_tmap_store_u8(&md, args.d, args.ldd * es, rows, depth, args.ldd * es, rows * args.ldd * es, 32);
    if (st != NVFP4_OK) return st;
  }
  auto kern = fp8_gemm_kernel<C>;
  st = allow_smem(reinterpret_cast<const void *>(kern), C::SMEM, dev.device);
  if (st != NVFP4_OK) return st;
  const int cluster = args.splits;
  int64_t grid = tiles * cluster;
  // split tiles: one per cluster (their partials are joined once); else persistent
  const int64_t cap = static_cast<int64_t>(dev.sm_count) * C::CTAS / cluster * cluster;
  if (args.splits == 1 && grid > cap) grid = cap;
  cudaError_t e = launch(kern, dim3(static_cast<unsigned>(grid)), dim3(C::THREADS), C::SMEM, (cudaStream_t)stream,
                         (flags & NVFP4_FLAG_PDL) != 0, cluster, mp, mq, md, args);
  return check_launch(e, name);
}

}  // namespace fp8
}  // namespace nvfp4
