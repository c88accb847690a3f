// Draw of one token per row of logits: temperature, top-k, top-p and min-p, from a given random
// number per row.
//
// For a row z with largest logit m, in fp32 (every step rounded to nearest):
//   x_i = (z_i - m) * (log2(e) / T),   e_i = 2^x_i,   w_i = rint(e_i * 2^30), a whole number
// Tokens are ordered by x, largest first, ties by index.  Every filter keeps a beginning of that order:
//   top-k  the first k;
//   top-p  those before which the tokens (of the k) weigh less than p times the k's total;
//   min-p  those with e_i >= min_p;
// and the first token always stays.  The token drawn is the first one, by index, at which the kept
// tokens' cumulative weight exceeds floor(u * total).  Sums of whole numbers are exact in any
// order, so the token depends neither on how a row is split over CTAs and threads nor on the order of
// atomics.  (A weight below 2^-31 of the largest is zero; 2^21 tokens of weight 2^30 stay below 2^53,
// so the products with p and u are taken in fp64 without losing a unit.)
//
// No sort.  A cluster of 1 to 8 CTAs owns a row; each of its warps owns a contiguous piece:
//   1. the row's maximum;
//   2. (top-k, top-p) counts and weights of 1024 classes of -x, each 1/32 wide, in shared memory; the
//      first CTA adds the others' and finds the class in which the k-th token, then p times the
//      total, is reached;
//   3. (top-k, top-p) that class's keys (the bits of -x, which order as -x does) go to a list in the first
//      CTA, which sorts it and reads off the cut: the last kept key and how many tokens that share
//      it are kept.  A class with more than kList tokens is first split again, by 256, down to a
//      single key if it must be (a row of equal logits needs no list at all);
//   4. the kept weight and the ties of every piece; then the piece that the random number falls in
//      is walked once more to the token.
// Without top-k and top-p only 1 and 4 run.  The row is read from memory once and then from L2.
#include <cuda_bf16.h>

#include "host.h"
#include "ptx.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;       // CTAs per row: the portable cluster size
constexpr int kClasses = 1024;    // classes of -x in [0, 32)
constexpr int kSplit = 256;       // parts of a class that is split again
constexpr int kList = 4096;       // keys sorted at once
constexpr int64_t kMaxVocab = 1 << 21;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kNoCut = 0xFFFFFFFFu;

struct SampleArgs {
  const void *logits;
  int64_t ld;
  int v, ctas;
  const float *uniform, *temperature;
  const int32_t *top_k;
  const float *top_p, *min_p;
  int32_t *tokens;
  float *logprobs;
};

// Where a sum reaches a target: class (or part) `bin`, with what the ones before it hold.
struct Found {
  uint32_t ok, bin, n, key, r;
  uint64_t count, mass;
};

struct Smem {
  uint64_t mass[kClasses];
  uint64_t part_mass[2][kSplit];
  uint32_t count[kClasses];
  uint32_t part_count[2][kSplit];
  uint32_t list[kList];
  uint32_t list_n[2];
  uint32_t base;
  Found found;
  float cta_max[kMaxCtas];
  uint64_t cta_mass[kMaxCtas];
  uint32_t cta_ties[kMaxCtas];
  float warp_max[kWarps];
  uint64_t warp_mass[kWarps];
  uint32_t warp_ties[kWarps];
  uint64_t scan[2][kWarps];
};

// A row as 16-byte vectors on 16-byte boundaries: the first may begin before the row and the last end
// after it; those two are read element by element.
template <typename T>
struct Row {
  static constexpr int EV = 16 / sizeof(T);
  const T *p;
  int off, v, vecs;
  __device__ __forceinline__ Row(const T *row, int n) : p(row), v(n) {
    off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    vecs = (off + n + EV - 1) / EV;
  }
  __device__ __forceinline__ void load(int vec, float (&f)[EV]) const {
    const int i0 = vec * EV - off;
    if (i0 >= 0 && i0 + EV <= v) {
      const uint4 q = *reinterpret_cast<const uint4 *>(p + i0);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) {
          f[2 * i] = __uint_as_float(w[i] << 16);
          f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
          f[i] = __uint_as_float(w[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < EV; ++i)
        f[i] = i0 + i >= 0 && i0 + i < v ? static_cast<float>(p[i0 + i]) : __uint_as_float(0xFF800000u);
    }
  }
};

// What turns a logit into its place in the order.
struct Scale {
  float m, c;
  bool only_max;  // only the logits equal to m have weight (m or c is infinite, or the row is greedy)
  // -x; tokens that weigh nothing (NaN included) come out at 32 or more, or as NaN
  __device__ __forceinline__ float neg_x(float z) const {
    if (only_max) return z == m ? 0.0f : 64.0f;
    return __fsub_rn(0.0f, __fmul_rn(__fsub_rn(z, m), c));
  }
};
__device__ __forceinline__ float exp2_neg(float nx) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-nx));
  return e;
}
__device__ __forceinline__ uint32_t weight_of(float e) { return __float2uint_rn(e * 1073741824.0f); }

// f(values of one vector) over the vectors [b, e) of a warp's piece, U vectors a lane in flight.
template <typename T, typename F>
__device__ __forceinline__ void walk(const Row<T> &row, int b, int e, int lane, F &&f) {
  constexpr int U = 4;
  for (int s = b + lane; s < e; s += 32 * U) {
    float z[U][Row<T>::EV];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + 32 * u < e) row.load(s + 32 * u, z[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + 32 * u < e) f(z[u]);
  }
}

__device__ __forceinline__ void row_sync(int ctas) {
  if (ctas > 1) cluster_sync();
  else __syncthreads();
}

// Exclusive prefix of (a, b) over the block's threads.
__device__ __forceinline__ void block_prefix(uint64_t (&scan)[2][kWarps], uint64_t &a, uint64_t &b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t na = __shfl_up_sync(0xFFFFFFFFu, ia, o), nb = __shfl_up_sync(0xFFFFFFFFu, ib, o);
    if (lane >= o) ia += na, ib += nb;
  }
  __syncthreads();
  if (lane == 31) scan[0][warp] = ia, scan[1][warp] = ib;
  __syncthreads();
  uint64_t pa = 0, pb = 0;
  for (int w = 0; w < warp; ++w) pa += scan[0][w], pb += scan[1][w];
  a = pa + ia - a;
  b = pb + ib - b;
}

// The bin of [0, n) in which the running count (or mass), starting from what found holds, reaches
// `target`; found then holds what lies before that bin.  Run by every thread of the first CTA.
__device__ void find_bin(Smem &s, const uint32_t *count, const uint64_t *mass, int n, bool by_mass, uint64_t target) {
  const uint64_t c0 = s.found.count, m0 = s.found.mass;
  const int per = n > kThreads ? n / kThreads : 1;
  const int b0 = threadIdx.x * per;
  uint64_t c = 0, m = 0;
  if (b0 < n)
    for (int i = 0; i < per; ++i) c += count[b0 + i], m += mass[b0 + i];
  block_prefix(s.scan, c, m);  // (its barriers come after every thread's read of found)
  if (threadIdx.x == 0) s.found.ok = 0;
  __syncthreads();
  c += c0;
  m += m0;
  if (b0 < n)
    for (int i = 0; i < per; ++i) {
      const uint64_t before = by_mass ? m : c, add = by_mass ? mass[b0 + i] : count[b0 + i];
      if (before < target && target <= before + add) {
        s.found.ok = 1;
        s.found.bin = b0 + i;
        s.found.n = count[b0 + i];
        s.found.count = c;
        s.found.mass = m;
      }
      c += count[b0 + i];
      m += mass[b0 + i];
    }
}

// Sorts the first CTA's list of n keys and finds the key at which the count (or mass) reaches
// `target`, how many of the tokens that share it are kept, and the mass up to there.
__device__ void find_key(Smem &s, int n, bool by_mass, uint64_t target) {
  int n2 = 32;
  while (n2 < n) n2 <<= 1;
  for (int i = n + threadIdx.x; i < n2; i += kThreads) s.list[i] = 0xFFFFFFFFu;
  __syncthreads();
  for (int k = 2; k <= n2; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < n2 / 2; i += kThreads) {
        const int a = 2 * i - (i & (j - 1)), b = a + j;
        const uint32_t x = s.list[a], y = s.list[b];
        if ((x > y) == ((a & k) == 0)) s.list[a] = y, s.list[b] = x;
      }
      __syncthreads();
    }
  const int per = (n + kThreads - 1) / kThreads, i0 = threadIdx.x * per;
  auto weight = [&](int i) { return static_cast<uint64_t>(weight_of(exp2_neg(__uint_as_float(s.list[i])))); };
  uint64_t c = 0, m = 0;
  for (int i = i0; i < i0 + per && i < n; ++i) ++c, m += weight(i);
  const uint64_t c0 = s.found.count, m0 = s.found.mass;
  block_prefix(s.scan, c, m);
  c += c0;
  m += m0;
  for (int i = i0; i < i0 + per && i < n; ++i) {
    const uint64_t w = weight(i), before = by_mass ? m : c;
    if (before < target && target <= before + (by_mass ? w : 1)) {
      const uint32_t key = s.list[i];
      int lo = 0, hi = i;  // first place of the key
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s.list[mid] < key) lo = mid + 1;
        else hi = mid;
      }
      s.found.key = key;
      s.found.r = i - lo + 1;
      s.found.mass = m + w;
    }
    ++c;
    m += w;
  }
}

// The kept beginning of the order: keys below `key`, and the first `r` tokens that have it.
struct Cut {
  uint32_t key, r;
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs p) {
  __shared__ Smem s;
  if (p.ctas > 1) cluster_arrive_relaxed();
  pdl_trigger();
  pdl_wait();
  const int ctas = p.ctas, rank = ctas > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t r = blockIdx.x / ctas;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Row<T> row(static_cast<const T *>(p.logits) + r * p.ld, p.v);
  constexpr int EV = Row<T>::EV;
  // this warp's vectors: pieces of equal length, in order over the cluster's warps
  const int piece = rank * kWarps + warp, pieces = ctas * kWarps;
  const int vb = static_cast<int>(static_cast<int64_t>(piece) * row.vecs / pieces);
  const int ve = static_cast<int>(static_cast<int64_t>(piece + 1) * row.vecs / pieces);

  const float t = p.temperature ? p.temperature[r] : 1.0f;
  const bool greedy = !(t > 0.0f);
  const int32_t k = p.top_k && !greedy ? p.top_k[r] : 0;
  const float top_p = p.top_p && !greedy ? p.top_p[r] : 1.0f;
  const float min_p = p.min_p && !greedy ? p.min_p[r] : 0.0f;
  const bool use_k = k > 0 && k < p.v, use_p = top_p < 1.0f;

  // 1. maximum (fmaxf passes over NaN)
  float mx = __uint_as_float(0xFF800000u);
  walk(row, vb, ve, lane, [&](const float(&z)[EV]) {
#pragma unroll
    for (int i = 0; i < EV; ++i) mx = fmaxf(mx, z[i]);
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  if (lane == 0) s.warp_max[warp] = mx;
  if (use_k || use_p) {
    for (int i = threadIdx.x; i < kClasses; i += kThreads) s.count[i] = 0, s.mass[i] = 0;
    for (int i = threadIdx.x; i < 2 * kSplit; i += kThreads) (&s.part_count[0][0])[i] = 0, (&s.part_mass[0][0])[i] = 0;
  }
  if (threadIdx.x == 0) {
    s.list_n[0] = s.list_n[1] = 0;
    s.found.count = s.found.mass = 0;
  }
  __syncthreads();
  mx = s.warp_max[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s.warp_max[w]);
  if (ctas > 1) {
    cluster_wait();  // every CTA of the row has started: its shared memory may be written
    if (threadIdx.x < ctas)
      st_cluster_u32(map_to_rank(smem_u32(&s.cta_max[rank]), threadIdx.x), __float_as_uint(mx));
    cluster_sync();
    mx = s.cta_max[0];
    for (int i = 1; i < ctas; ++i) mx = fmaxf(mx, s.cta_max[i]);
  }
  if (mx == __uint_as_float(0xFF800000u)) {  // nothing but -inf and NaN (the same on every CTA of the row)
    if (rank == 0 && threadIdx.x == 0) {
      p.tokens[r] = -1;
      if (p.logprobs) p.logprobs[r] = mx;
    }
    return;
  }
  const float c = greedy ? 1.0f : __fdiv_rn(kLog2e, t);
  const float inf = __uint_as_float(0x7F800000u);
  const Scale sc{mx, c, greedy || mx == inf || c == inf};
  Cut cut{kNoCut, 0};

  // 2. and 3. the cut of top-k and top-p
  if (use_k || use_p) {
    walk(row, vb, ve, lane, [&](const float(&z)[EV]) {
#pragma unroll
      for (int i = 0; i < EV; ++i) {
        const float nx = sc.neg_x(z[i]);
        if (nx < 32.0f) {
          const int b = static_cast<int>(nx * 32.0f);
          atomicAdd(&s.count[b], 1u);
          if (use_p) atomicAdd(reinterpret_cast<unsigned long long *>(&s.mass[b]),
                               static_cast<unsigned long long>(weight_of(exp2_neg(nx))));
        }
      }
    });
    __syncthreads();
    if (rank != 0)
      for (int i = threadIdx.x; i < kClasses; i += kThreads)
        if (s.count[i]) {
          red_add_cluster_u32(map_to_rank(smem_u32(&s.count[i]), 0), s.count[i]);
          if (use_p) red_add_cluster_u64(map_to_rank(smem_u32(&s.mass[i]), 0), s.mass[i]);
        }
    row_sync(ctas);
    int level = 0;  // splits made so far: they alternate between two sets of bins
    const uint32_t found0 = map_to_rank(smem_u32(&s.found), 0);
    auto found_u32 = [&](size_t off) { return ld_cluster_u32(found0 + static_cast<uint32_t>(off)); };
    auto found_u64 = [&](size_t off) { return ld_cluster_u64(found0 + static_cast<uint32_t>(off)); };
    // Keeps the shortest beginning of the order whose count (or mass) reaches target; returns its mass.
    // Every branch goes by what the first CTA found, so all CTAs of the row take it alike.
    auto keep = [&](bool by_mass, uint64_t target, int which) -> uint64_t {
      if (rank == 0) {
        if (threadIdx.x == 0) s.found.count = s.found.mass = 0;
        __syncthreads();
        find_bin(s, s.count, s.mass, kClasses, by_mass, target);
      }
      row_sync(ctas);
      if (!found_u32(offsetof(Found, ok))) return 0;  // fewer tokens have weight: nothing to cut
      const uint32_t bin = found_u32(offsetof(Found, bin));
      uint32_t lo = __float_as_uint(static_cast<float>(bin) / 32.0f), hi = __float_as_uint(static_cast<float>(bin + 1) / 32.0f);
      uint32_t n = found_u32(offsetof(Found, n));
      while (n > kList && hi - lo > 1) {
        const int buf = level++ & 1;
        int shift = 0;
        while (((hi - lo - 1) >> shift) >= kSplit) ++shift;
        walk(row, vb, ve, lane, [&](const float(&z)[EV]) {
#pragma unroll
          for (int i = 0; i < EV; ++i) {
            const float nx = sc.neg_x(z[i]);
            const uint32_t key = __float_as_uint(nx);
            if (nx < 32.0f && key >= lo && key < hi) {
              atomicAdd(&s.part_count[buf][(key - lo) >> shift], 1u);
              atomicAdd(reinterpret_cast<unsigned long long *>(&s.part_mass[buf][(key - lo) >> shift]),
                        static_cast<unsigned long long>(weight_of(exp2_neg(nx))));
            }
          }
        });
        __syncthreads();
        for (int i = threadIdx.x; i < kSplit; i += kThreads) {
          if (rank != 0 && s.part_count[buf][i]) {
            red_add_cluster_u32(map_to_rank(smem_u32(&s.part_count[buf][i]), 0), s.part_count[buf][i]);
            red_add_cluster_u64(map_to_rank(smem_u32(&s.part_mass[buf][i]), 0), s.part_mass[buf][i]);
          }
          s.part_count[buf ^ 1][i] = 0;  // (nobody adds to it before the next barrier)
          s.part_mass[buf ^ 1][i] = 0;
        }
        row_sync(ctas);
        if (rank == 0) find_bin(s, s.part_count[buf], s.part_mass[buf], kSplit, by_mass, target);
        row_sync(ctas);
        lo += found_u32(offsetof(Found, bin)) << shift;
        hi = min(hi, lo + (1u << shift));
        n = found_u32(offsetof(Found, n));
      }
      Cut got;
      uint64_t mass;
      if (hi - lo == 1) {
        const uint64_t w = weight_of(exp2_neg(__uint_as_float(lo))), m0 = found_u64(offsetof(Found, mass));
        const uint64_t before = by_mass ? m0 : found_u64(offsetof(Found, count)), each = by_mass ? w : 1;
        got = Cut{lo, static_cast<uint32_t>((target - before + each - 1) / each)};
        mass = m0 + got.r * w;
        row_sync(ctas);  // everyone has read found
      } else {
        walk(row, vb, ve, lane, [&](const float(&z)[EV]) {
#pragma unroll
          for (int i = 0; i < EV; ++i) {
            const float nx = sc.neg_x(z[i]);
            const uint32_t key = __float_as_uint(nx);
            if (nx < 32.0f && key >= lo && key < hi) s.list[atomicAdd(&s.list_n[which], 1u)] = key;
          }
        });
        __syncthreads();
        if (rank != 0) {
          const uint32_t mine = s.list_n[which];
          if (threadIdx.x == 0 && mine) s.base = atom_add_cluster_u32(map_to_rank(smem_u32(&s.list_n[which]), 0), mine);
          __syncthreads();
          for (uint32_t i = threadIdx.x; i < mine; i += kThreads)
            st_cluster_u32(map_to_rank(smem_u32(&s.list[s.base + i]), 0), s.list[i]);
        }
        row_sync(ctas);
        if (rank == 0) find_key(s, static_cast<int>(n), by_mass, target);
        row_sync(ctas);
        got = Cut{found_u32(offsetof(Found, key)), found_u32(offsetof(Found, r))};
        mass = found_u64(offsetof(Found, mass));
        row_sync(ctas);  // everyone has read found
      }
      if (got.key < cut.key || (got.key == cut.key && got.r < cut.r)) cut = got;
      return mass;
    };
    uint64_t total = 0;
    if (use_k) total = keep(false, static_cast<uint64_t>(k), 0);
    if (use_p) {
      if (total == 0) {  // no top-k, or fewer than k tokens have weight: the whole row's mass
        if (rank == 0) {
          uint64_t a = 0, b = 0;
          for (int i = threadIdx.x; i < kClasses; i += kThreads) a += s.mass[i];
          const uint64_t own = a;
          block_prefix(s.scan, a, b);
          if (threadIdx.x == kThreads - 1) s.found.mass = a + own;
        }
        row_sync(ctas);
        total = found_u64(offsetof(Found, mass));
        row_sync(ctas);
      }
      const double want = ceil(static_cast<double>(top_p) * static_cast<double>(total));
      keep(true, want < 1.0 ? 1 : static_cast<uint64_t>(want), 1);
    }
  }
  // the first of the order stays whatever the filters say
  if (greedy || min_p > 1.0f || min_p != min_p) cut = Cut{0, 1};

  // 4. kept weight and ties of every piece
  uint64_t mass = 0;
  uint32_t ties = 0;
  walk(row, vb, ve, lane, [&](const float(&z)[EV]) {
#pragma unroll
    for (int i = 0; i < EV; ++i) {
      const float nx = sc.neg_x(z[i]);
      const uint32_t key = __float_as_uint(nx);
      if (nx < 32.0f && key <= cut.key) {
        const float e = exp2_neg(nx);
        if (e >= min_p) {
          if (key == cut.key) ++ties;
          else mass += weight_of(e);
        }
      }
    }
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mass += __shfl_xor_sync(0xFFFFFFFFu, mass, o);
    ties += __shfl_xor_sync(0xFFFFFFFFu, ties, o);
  }
  if (lane == 0) s.warp_mass[warp] = mass, s.warp_ties[warp] = ties;
  __syncthreads();
  uint64_t cta_mass = 0;
  uint32_t cta_ties = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) cta_mass += s.warp_mass[w], cta_ties += s.warp_ties[w];
  if (ctas > 1) {
    if (threadIdx.x < ctas) {
      st_cluster_u64(map_to_rank(smem_u32(&s.cta_mass[rank]), threadIdx.x), cta_mass);
      st_cluster_u32(map_to_rank(smem_u32(&s.cta_ties[rank]), threadIdx.x), cta_ties);
    }
    cluster_sync();  // (the last access to another CTA's shared memory: a CTA may leave after it)
  } else if (threadIdx.x == 0) {
    s.cta_mass[0] = cta_mass;
    s.cta_ties[0] = cta_ties;
  }
  if (ctas == 1) __syncthreads();
  const uint64_t wc = cut.key == kNoCut ? 0 : weight_of(exp2_neg(__uint_as_float(cut.key)));
  uint64_t total = 0;
  uint32_t all_ties = 0;
  for (int i = 0; i < ctas; ++i) total += s.cta_mass[i], all_ties += s.cta_ties[i];
  total += wc * min(all_ties, cut.r);
  const double want = static_cast<double>(p.uniform[r]) * static_cast<double>(total);
  uint64_t target = want > 0.0 ? static_cast<uint64_t>(want) : 0;
  if (target >= total) target = total - 1;
  // the piece that holds it: ties are kept by index until r of them are
  uint32_t left = cut.r;  // ties still to keep
  uint64_t before = 0;
  bool mine = false;
  for (int i = 0; i <= rank; ++i) {
    const uint32_t kept = min(left, s.cta_ties[i]);
    const uint64_t held = s.cta_mass[i] + wc * kept;
    if (i == rank) {
      mine = target >= before && target < before + held;
    } else {
      before += held;
      left -= kept;
    }
  }
  if (!mine) return;
  for (int w = 0; w <= warp; ++w) {
    const uint32_t kept = min(left, s.warp_ties[w]);
    const uint64_t held = s.warp_mass[w] + wc * kept;
    if (w == warp) {
      mine = target >= before && target < before + held;
    } else {
      before += held;
      left -= kept;
    }
  }
  if (!mine) return;
  // (one warp of the row is left) walk its piece to the token
  for (int v0 = vb; v0 < ve; v0 += 32) {
    float z[EV];
    uint32_t wt[EV];
    uint32_t n_ties = 0;
    const bool in = v0 + lane < ve;
    if (in) row.load(v0 + lane, z);
    uint32_t tie_mask = 0;
#pragma unroll
    for (int i = 0; i < EV; ++i) {
      wt[i] = 0;
      if (!in) continue;
      const float nx = sc.neg_x(z[i]);
      const uint32_t key = __float_as_uint(nx);
      if (nx < 32.0f && key <= cut.key) {
        const float e = exp2_neg(nx);
        if (e >= min_p) {
          wt[i] = weight_of(e);
          if (key == cut.key) tie_mask |= 1u << i, ++n_ties;
        }
      }
    }
    uint32_t tb = n_ties;  // ties before this lane's vector
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t n = __shfl_up_sync(0xFFFFFFFFu, tb, o);
      if (lane >= o) tb += n;
    }
    const uint32_t step_ties = __shfl_sync(0xFFFFFFFFu, tb, 31);
    tb -= n_ties;
    uint64_t held = 0;
#pragma unroll
    for (int i = 0; i < EV; ++i) {
      if (tie_mask >> i & 1) {
        if (tb >= left) wt[i] = 0;
        ++tb;
      }
      held += wt[i];
    }
    uint64_t upto = held;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t n = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += n;
    }
    const uint64_t step = __shfl_sync(0xFFFFFFFFu, upto, 31);
    if (target < before + step) {
      uint64_t at = before + upto - held;
      if (target >= at && target < at + held) {
#pragma unroll
        for (int i = 0; i < EV; ++i) {
          if (target >= at && target < at + wt[i]) {
            p.tokens[r] = (v0 + lane) * EV + i - row.off;
            if (p.logprobs)
              p.logprobs[r] = __fsub_rn(__fmul_rn(-sc.neg_x(z[i]), 0.6931471805599453f),
                                        logf(__fmul_rn(__ull2float_rn(total), 1.0f / 1073741824.0f)));
          }
          at += wt[i];
        }
      }
      return;
    }
    before += step;
    left -= min(left, step_ties);
  }
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status_t sample_tokens(const void *logits, int logits_type, int64_t ld, const float *uniform,
                                        const float *temperature, const int32_t *top_k, const float *top_p,
                                        const float *min_p, int32_t *tokens, float *logprobs, int64_t rows, int64_t vocab,
                                        uint32_t flags, nvfp4_stream_t stream) {
  clear_error();
  const char *name = "sample_tokens";
  if (rows < 0 || vocab <= 0 || rows >= (1LL << 28))
    return fail(NVFP4_ERR_INVALID_ARG, "%s: rows=%lld vocab=%lld", name, (long long)rows, (long long)vocab);
  if (vocab > kMaxVocab)
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: vocab=%lld (at most %lld)", name, (long long)vocab, (long long)kMaxVocab);
  if (logits_type != NVFP4_DTYPE_BF16 && logits_type != NVFP4_DTYPE_F32)
    return fail(NVFP4_ERR_INVALID_ARG, "%s: logits_type=%d", name, logits_type);
  if (flags & ~(uint32_t)NVFP4_FLAG_PDL) return fail(NVFP4_ERR_INVALID_ARG, "%s: unknown flags 0x%x", name, flags);
  if (ld != 0 && ld < vocab)
    return fail(NVFP4_ERR_INVALID_ARG, "%s: ld=%lld < vocab=%lld", name, (long long)ld, (long long)vocab);
  if (rows == 0) return NVFP4_OK;
  if (!logits || !uniform || !tokens) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", name);
  const bool f32 = logits_type == NVFP4_DTYPE_F32;
  if (!aligned(logits, f32 ? 4 : 2) || !aligned(uniform, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
      !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4) || !aligned(logprobs, 4))
    return fail(NVFP4_ERR_MISALIGNED, "%s: a pointer is not aligned to its element", name);
  DeviceInfo dev;
  nvfp4_status_t st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  // CTAs per row: as many as give every SM two CTAs, while each still has 2048 tokens to read
  int ctas = 1;
  while (ctas < kMaxCtas && rows * ctas * 2 <= 2LL * dev.sm_count && vocab >= 2048LL * 2 * ctas) ctas *= 2;
  SampleArgs a{logits, ld, static_cast<int>(vocab), ctas, uniform, temperature, top_k, top_p, min_p, tokens, logprobs};
  auto kern = f32 ? sample_kernel<float> : sample_kernel<__nv_bfloat16>;
  return check_launch(launch(kern, dim3(static_cast<unsigned>(rows * ctas)), dim3(kThreads), 0, (cudaStream_t)stream,
                             (flags & NVFP4_FLAG_PDL) != 0, ctas, a), name);
}
