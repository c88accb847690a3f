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
// atomics.  (A weight below 2^-31 of the largest is zero; 2^21 tokens of weight 2^30 stay below 2^53, so a total is
// exact in fp64, and its products with p and u are rounded once.)
//
// No sort of the row.  A cluster of 1 to 8 CTAs owns a row; each of its warps owns a contiguous piece:
//   1. the row's maximum (and the largest logits of each thread's two heaviest vectors);
//   2. (top-k, top-p) a bracket of -x that the cut must fall in:
//      top-k  the threads' maxima are tokens, so the k-th largest of them bounds the k-th token
//             from below: everything from there up is the bracket;
//      top-p  the threads' maxima, which hold the heavy tokens, and a histogram of every eighth vector
//             of the rest estimate where the mass reaches p; the bracket is 4.5 standard deviations
//             either way;
//   3. one pass that adds up the weight above the bracket (top-p; with top-k nothing is above) and
//      keeps the logits inside it in a list per thread;
//   4. the cut: the last kept key (the bits of -x, which order as -x does) and how many tokens that share
//      it are kept.  The bracket is split by 256 until at most kFew keys are left; the first CTA compares
//      those with one another;
//   5. the kept weight and the ties of every piece, from the weight above and the lists; then the piece
//      that the random number falls in is split over its CTA's warps, and one of them walks its
//      part to the token.
// Where the bracket is missed or a list overflows (equal logits, k or p near the end of a flat row, top-p over
// 131072 and more fp32 logits in one CTA: a list holds half as many of them) the
// cut is found from the row itself: counts and weights of 1024 classes of -x, then splits of the class
// down to a single key if need be (a row of equal logits), with a pass over the row each, and one more
// pass for 5.  Both ways give the same cut.  Without top-k and top-p only 1 and 5 run, from the row.
//
// The row is read from memory once, then from L2.  What bounds it, measured on device: 256 rows of 131072
// bf16 with top-p take 70 us (floor 10 us, the logits read once), of them 6 the maximum, 8 the bracket, 18 to
// 26 the pass (issue: about 15 instructions a token on the SMs that hold two rows), 10 the cut; 64 rows with
// every filter 28 us (floor 2.5) and one row of 32000 fp32 7.6 us, which is latency: seven passes or
// cluster barriers of one to three microseconds each.  Between the steps of a decoder the code itself
// leaves L2, and fetching it costs as much again (one row: 19 us with nothing in L2, 27 us before the
// code was halved: 304 -> 155 KB).
// Measured and not kept: classes and 64-bit masses of the whole row with shared-memory atomics, two of
// them a token (328 and 83 us: a 64-bit one costs several 32-bit ones), which is now only the fallback;
// a sample of every fourth vector with p (1 - p) for the variance, which overflowed lists (206 us); a
// sorted list instead of keys compared with one another (33 -> 26 us at 64 rows); find_bin and find_key
// as calls (64 rows 28 -> 32 us).
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
constexpr int kFew = 256;         // keys compared with one another
constexpr int kListBytes = 128;   // a thread's list of the bracket's logits: 64 of bf16, 32 of fp32
constexpr int kSampled = 8;       // the top-p bracket is estimated from every eighth group of vectors
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

// Weight that top-p's tokens must reach: those before a kept token weigh less than top_p * total.
__device__ __forceinline__ uint64_t mass_target(float top_p, uint64_t total) {
  const double want = ceil(static_cast<double>(top_p) * static_cast<double>(total));
  return want < 1.0 ? 1 : static_cast<uint64_t>(want);
}

// Where a sum reaches a target: class (or part) `bin`, with what the ones before it hold.
struct Found {
  uint32_t ok, bin, n, key, r;
  uint64_t count, mass;
};

struct Smem {
  uint32_t kept[kListBytes / 4 * kThreads];
  uint64_t mass[kClasses];
  uint64_t part_mass[2][kSplit];
  uint32_t count[kClasses];
  uint32_t part_count[2][kSplit];
  uint32_t part_lo[kSplit], part_hi[kSplit];
  uint2 few[kFew];  // key, weight
  uint32_t few_n[2];
  uint32_t base;
  Found found;
  // the bracket's edges in classes, and what the cluster found of it
  uint32_t edge_lo, edge_hi, bracket_n, overflow;
  uint32_t vectors, sampled;  // of the row, and in the sample
  uint64_t bracket_mass, above, total;
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
  static constexpr int kList = kListBytes / sizeof(T);
  const T *p;
  int off, v, vecs;
  __device__ __forceinline__ Row(const T *row, int n) : p(row), v(n) {
    off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    vecs = (off + n + EV - 1) / EV;
  }
  // Vector `vec` as it lies in memory; places outside the row hold -inf.
  __device__ __forceinline__ uint4 load(int vec) const {
    const int i0 = vec * EV - off;
    if (i0 >= 0 && i0 + EV <= v) return *reinterpret_cast<const uint4 *>(p + i0);
    return load_edge(p, i0, v);
  }
  static __device__ __noinline__ uint4 load_edge(const T *p, int i0, int v) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < EV; ++i) {
      const bool in = i0 + i >= 0 && i0 + i < v;
      if constexpr (sizeof(T) == 2) {
        const uint32_t h = in ? __bfloat16_as_ushort(p[i0 + i]) : 0xFF80u;
        w[i / 2] |= h << (16 * (i & 1));
      } else {
        w[i] = in ? __float_as_uint(p[i0 + i]) : 0xFF800000u;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ void unpack(const uint4 &q, float (&f)[EV]) {
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
  }
  // Largest value of a vector (NaN passed over).
  static __device__ __forceinline__ float max_of(const uint4 &q) {
    if constexpr (sizeof(T) == 2) {
      auto max2 = [](uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
      };
      const uint32_t m = max2(max2(q.x, q.y), max2(q.z, q.w));
      return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    } else {
      return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)), fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
    }
  }
};

// What turns a logit into its place in the order.
struct Scale {
  float m, c;
  // -x = (m - z) c, which is the exact negative of (z - m) c.  It is never -0, whose bits are no key below
  // any edge: m is not -0, so m - z is +0 for either zero z.  A token whose -x is 32 or more, or NaN, weighs
  // nothing (exp2_neg and weight_of give 0 for those too).
  __device__ __forceinline__ float neg_x(float z) const { return __fmul_rn(__fsub_rn(m, z), c); }
  // Two at once: z * -1 + m rounds as m - z does.
  __device__ __forceinline__ void neg_x2(float z0, float z1, float (&nx)[2]) const {
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 d, {%5, %5};\n"
        " fma.rn.f32x2 a, a, b, d;\n mov.b64 b, {%6, %6};\n mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
        : "=f"(nx[0]), "=f"(nx[1])
        : "f"(z0), "f"(z1), "f"(-1.0f), "f"(m), "f"(c));
  }
};
__device__ __forceinline__ float exp2_neg(float nx) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-nx));
  return e;
}
__device__ __forceinline__ uint32_t weight_of(float e) { return __float2uint_rn(e * 1073741824.0f); }

// f(vector, its index) over the vectors b + lane, b + lane + 32 * STEP, ... of [b, e), U of them in flight (one where speed does not count: code is kept small, since a step of a
// decoder finds it in DRAM again).
template <int STEP, int U, typename T, typename F>
__device__ __forceinline__ void walk(const Row<T> &row, int b, int e, int lane, F &&f) {
  for (int s = b + lane; s < e; s += 32 * STEP * U) {
    uint4 q[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + 32 * STEP * u < e) q[u] = row.load(s + 32 * STEP * u);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + 32 * STEP * u < e) f(q[u], s + 32 * STEP * u);
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
__device__ __forceinline__ void find_bin(Smem &s, const uint32_t *count, const uint64_t *mass, int n, bool by_mass, uint64_t target) {
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

// The cut among the first CTA's n <= kFew keys, each compared with all others (fewer instructions than
// sorting them, and no barriers): the key at which the count reaches `k` (0: no such target), then
// the one at which the mass reaches `target`, or with top_p < 1 that share of the mass up to the first cut.
// Run by every thread of the first CTA.
__device__ __forceinline__ void find_key(Smem &s, int n, uint64_t k, uint64_t target, float top_p) {
  uint32_t key = 0, w = 0, eq = 0;
  uint64_t less = s.found.count, mass = s.found.mass;
  const bool in = static_cast<int>(threadIdx.x) < n;
  if (in) {
    key = s.few[threadIdx.x].x;
    w = weight_of(exp2_neg(__uint_as_float(key)));
    s.few[threadIdx.x].y = w;
  }
  __syncthreads();
  if (in)
    for (int j = 0; j < n; ++j) {
      const uint2 o = s.few[j];
      if (o.x < key) ++less, mass += o.y;
      eq += o.x == key;
    }
  if (k > 0) {
    if (in && less < k && k <= less + eq) {  // (tokens that share the key write the same)
      s.found.key = key;
      s.found.r = static_cast<uint32_t>(k - less);
      s.found.mass = mass + (k - less) * w;
    }
    __syncthreads();
    if (top_p >= 1.0f) return;
    target = mass_target(top_p, s.found.mass);
    __syncthreads();
  }
  if (in && mass < target && target <= mass + static_cast<uint64_t>(eq) * w) {
    s.found.key = key;
    s.found.r = static_cast<uint32_t>((target - mass + w - 1) / w);
  }
}

// The kept beginning of the order: keys below `key`, and the first `r` tokens that have it.
struct Cut {
  uint32_t key, r;
};

// The bracket of a top-p cut, run by every thread of the first CTA: classes below edge_lo lie above the
// cut, classes from edge_hi on below it, to 4.5 standard deviations.  s.count holds the sampled tokens
// (taken at their class's middle; one stands for k = s.vectors / s.sampled), s.mass the weights of the
// thread maxima, which the sample leaves out: a heavy token that one sample holds and the next does not
// would blur everything.  The estimated share of the mass above a cut at share p has variance
//   ((1 - p)^2 sum of w^2 above + p^2 sum of w^2 below) k (k - 1) / (sum of w)^2
// over the tokens that were sampled.  The classes' own width adds a little (0.01 p (1 - p)).
// `most`: keys that the lists should have to hold at most.
__device__ __forceinline__ void sample_bracket(Smem &s, float top_p, float most) {
  constexpr int PER = kClasses / kThreads;
  const int b0 = threadIdx.x * PER;
  uint64_t c = 0, m = 0, sq = 0, zero = 0;
  const float k = static_cast<float>(s.vectors) / static_cast<float>(s.sampled);
  const uint64_t k256 = static_cast<uint64_t>(k * 256.0f + 0.5f);
  auto weight = [&](int b) { return static_cast<uint64_t>(weight_of(exp2_neg((b + 0.5f) / 32.0f))); };
  auto mass = [&](int b) { return (s.count[b] * weight(b) * k256 >> 8) + s.mass[b]; };
  auto square = [&](int b) { return s.count[b] * (weight(b) * weight(b) >> 14); };  // in units of 2^14
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c += s.count[b0 + i];
    m += mass(b0 + i);
    sq += square(b0 + i);
  }
  const uint64_t own_m = m, own_sq = sq;
  block_prefix(s.scan, c, m);
  block_prefix(s.scan, sq, zero);
  __syncthreads();
  if (threadIdx.x == kThreads - 1) s.total = m + own_m, s.above = sq + own_sq;
  if (threadIdx.x == 0) s.edge_lo = 0, s.edge_hi = kClasses, s.bracket_n = 0, s.bracket_mass = 0;
  __syncthreads();
  const float total = static_cast<float>(s.total), all_sq = static_cast<float>(s.above);
  // the first class of this thread's that ends past `x`: f(class, tokens before it, squares up to its end)
  auto crossing = [&](float x, auto &&f) {
    uint64_t ci = c, mi = m, si = sq;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float before = static_cast<float>(mi);
      mi += mass(b0 + i);
      si += square(b0 + i);
      if (before <= x && static_cast<float>(mi) > x) f(b0 + i, ci, si);
      ci += s.count[b0 + i];
    }
  };
  crossing(top_p * total, [&](int, uint64_t, uint64_t si) { s.bracket_mass = si; });
  __syncthreads();
  const float up = static_cast<float>(s.bracket_mass), q = 1.0f - top_p;
  const float var = (q * q * up + top_p * top_p * fmaxf(all_sq - up, 0.0f)) * 16384.0f / (total * total);
  const float width = 4.5f * sqrtf(fmaxf(var * k * (k - 1.0f), 0.0f)) + 0.01f * q * top_p;
  crossing((top_p - width) * total, [&](int b, uint64_t ci, uint64_t) { s.edge_lo = b, s.bracket_n = static_cast<uint32_t>(ci); });
  __syncthreads();
  const int lo = static_cast<int>(s.edge_lo);
  const float to = (top_p + width) * total, n0 = static_cast<float>(s.bracket_n);
#pragma unroll
  for (int i = 0; i < PER; ++i) {  // the last class it needs, or the last that fits
    m += mass(b0 + i);
    c += s.count[b0 + i];
    if (b0 + i >= lo && (static_cast<float>(m) >= to || (static_cast<float>(c) - n0) * k >= most))
      atomicMin(&s.edge_hi, static_cast<uint32_t>(b0 + i + 1));
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem &s = *reinterpret_cast<Smem *>(smem_raw);
  if (p.ctas > 1) cluster_arrive_relaxed();
  pdl_trigger();
  pdl_wait();
  const int ctas = p.ctas, rank = ctas > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t r = blockIdx.x / ctas;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Row<T> row(static_cast<const T *>(p.logits) + r * p.ld, p.v);
  constexpr int EV = Row<T>::EV;
  const float inf = __uint_as_float(0x7F800000u);
  // this warp's vectors: pieces of equal length, in order over the cluster's warps
  const int pieces = ctas * kWarps;
  auto piece_at = [&](int i) { return static_cast<int>(static_cast<int64_t>(i) * row.vecs / pieces); };
  const int vb = piece_at(rank * kWarps + warp), ve = piece_at(rank * kWarps + warp + 1);

  const float t = p.temperature ? p.temperature[r] : 1.0f;
  const bool greedy = !(t > 0.0f);
  // greedy, or a min_p that no token passes: the first of the order alone, whatever the other filters say
  const bool only_first = greedy || (p.min_p && !(p.min_p[r] <= 1.0f));
  const int32_t k = p.top_k && !only_first ? p.top_k[r] : 0;
  const float top_p = p.top_p && !only_first ? p.top_p[r] : 1.0f;
  const float min_p = p.min_p && !only_first ? p.min_p[r] : 0.0f;
  const bool use_k = k > 0 && k < p.v, use_p = top_p < 1.0f;

  // 1. maximum; m1 and m2: the largest logits of this thread's two heaviest vectors, i1 and i2
  float m1 = -inf, m2 = -inf;
  int i1 = 0, i2 = 0;
  walk<1, 4>(row, vb, ve, lane, [&](const uint4 &q, int i) {
    const float v = Row<T>::max_of(q);
    const bool first = v > m1, second = v > m2;
    m2 = first ? m1 : second ? v : m2;
    i2 = first ? i1 : second ? i : i2;
    m1 = first ? v : m1;
    i1 = first ? i : i1;
  });
  float mx = m1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  if (lane == 0) s.warp_max[warp] = mx;
  auto clear_classes = [&]() {
    for (int i = threadIdx.x; i < kClasses; i += kThreads) s.count[i] = 0, s.mass[i] = 0;
  };
  if (use_k || use_p) {
    clear_classes();
    for (int i = threadIdx.x; i < 2 * kSplit; i += kThreads) (&s.part_count[0][0])[i] = 0, (&s.part_mass[0][0])[i] = 0;
  }
  if (threadIdx.x < kSplit) s.part_lo[threadIdx.x] = s.part_hi[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    s.few_n[0] = s.few_n[1] = 0;
    s.found.count = s.found.mass = 0;
    s.vectors = s.sampled = 0;
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
  mx = __fadd_rn(mx, 0.0f);  // -0 becomes +0 (see Scale)
  if (mx == -inf) {  // nothing but -inf and NaN (the same on every CTA of the row)
    if (rank == 0 && threadIdx.x == 0) {
      p.tokens[r] = -1;
      if (p.logprobs) p.logprobs[r] = mx;
    }
    return;
  }
  // Only the logits equal to the largest have weight where that or the factor is infinite, or the row is
  // greedy: they become 0 and the others -inf.
  const float c0 = greedy ? 1.0f : __fdiv_rn(kLog2e, t);
  const bool only_max = greedy || mx == inf || c0 == inf;
  const Scale sc{only_max ? 0.0f : mx, only_max ? 1.0f : c0};
  auto unpack = [&](const uint4 &q, float(&z)[EV]) {
    Row<T>::unpack(q, z);
    if (only_max)
#pragma unroll
      for (int i = 0; i < EV; ++i) z[i] = z[i] == mx ? 0.0f : -inf;
  };
  Cut cut{kNoCut, 0};
  // What this thread saw above the bracket, and how many keys it keeps of the bracket itself.
  uint64_t above = 0;
  int mine = 0;
  bool listed = false;
  T *const list = reinterpret_cast<T *>(s.kept) + threadIdx.x;  // entry i at i * kThreads

  if (use_k || use_p) {
    auto to_first = [&](const void *q) { return map_to_rank(smem_u32(q), 0); };
    // Adds this CTA's bins to the first CTA's.
    auto add_to_first = [&](uint32_t *count, uint64_t *mass, int n) {
      if (rank != 0)
        for (int i = threadIdx.x; i < n; i += kThreads) {
          if (count[i]) red_add_cluster_u32(to_first(&count[i]), count[i]);
          if (mass[i]) red_add_cluster_u64(to_first(&mass[i]), mass[i]);
        }
    };
    auto class_edge = [](uint32_t b) { return static_cast<float>(b) / 32.0f; };
    // Reads a field of the first CTA's shared memory.
    auto first_u32 = [&](const uint32_t &f) { return ctas > 1 ? ld_cluster_u32(to_first(&f)) : f; };
    auto first_u64 = [&](const uint64_t &f) { return ctas > 1 ? ld_cluster_u64(to_first(&f)) : f; };

    // 2. the bracket
    // a thread maximum is one token, counted for top-k and weighed for top-p (the halves of the weights' sums
    // in the lists' room, which is not in use yet: 1024 maxima a CTA cannot overflow them)
    uint32_t *const half = s.kept;
    if (!use_k) {
      for (int i = threadIdx.x; i < 2 * kClasses; i += kThreads) half[i] = 0;
      __syncthreads();
    }
    auto count_max = [&](float z, int i) {
      const float nx = sc.neg_x(only_max ? (z == mx ? 0.0f : -inf) : z);
      if (!(nx < 32.0f)) return;
      const int b = static_cast<int>(nx * 32.0f);
      if (use_k) {
        atomicAdd(&s.count[b], 1u);
      } else {
        const uint32_t w = weight_of(exp2_neg(nx));
        atomicAdd(&half[b], w & 0xFFFFu);
        atomicAdd(&half[kClasses + b], w >> 16);
        // the sample below counts it too if it holds its vector
        if (((i - vb - lane) >> 5) % kSampled == 0) atomicSub(&s.count[b], 1u);
      }
    };
    count_max(m1, i1);
    count_max(m2, i2);
    if (!use_k) {
      if (lane == 0) {  // groups of 32 vectors, every kSampled-th of them in the sample
        const int len = ve - vb, groups = len / (32 * kSampled), rest = len - groups * 32 * kSampled;
        red_add_cluster_u32(to_first(&s.vectors), static_cast<uint32_t>(len));
        red_add_cluster_u32(to_first(&s.sampled), static_cast<uint32_t>(groups * 32 + min(rest, 32)));
      }
      walk<kSampled, 4>(row, vb, ve, lane, [&](const uint4 &q, int) {
        float z[EV];
        unpack(q, z);
#pragma unroll
        for (int i = 0; i < EV; ++i) {
          const float nx = sc.neg_x(z[i]);
          if (nx < 32.0f) atomicAdd(&s.count[static_cast<int>(nx * 32.0f)], 1u);
        }
      });
    }
    __syncthreads();
    if (!use_k) {
      for (int i = threadIdx.x; i < kClasses; i += kThreads)
        if (half[i] | half[kClasses + i])  // (added, not stored: the first CTA's may be getting others' already)
          red_add_cluster_u64(map_to_rank(smem_u32(&s.mass[i]), rank), (static_cast<uint64_t>(half[kClasses + i]) << 16) + half[i]);
      __syncthreads();
    }
    add_to_first(s.count, s.mass, kClasses);
    row_sync(ctas);
    if (rank == 0) {
      if (use_k) {
        find_bin(s, s.count, s.mass, kClasses, false, static_cast<uint64_t>(k));
        __syncthreads();
        if (threadIdx.x == 0) s.edge_lo = 0, s.edge_hi = s.found.ok ? s.found.bin + 1 : 0;
      } else {
        sample_bracket(s, top_p, 0.5f * Row<T>::kList * kThreads * ctas);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        s.bracket_n = s.overflow = 0;
        s.bracket_mass = s.above = s.total = 0;
      }
    }
    row_sync(ctas);
    const uint32_t edge_lo = first_u32(s.edge_lo), edge_hi = first_u32(s.edge_hi);
    uint32_t n = 0;        // keys in the bracket
    uint64_t total = 0;    // top-p without top-k: the row's mass
    if (edge_hi > edge_lo) {
      // 3. what is above the bracket, and the keys inside it
      const float lo = class_edge(edge_lo), hi = class_edge(edge_hi);
      uint64_t all = 0;
      // `mine` past the list's end says that it overflowed
      T *at = list;
      auto room = [&]() {
        if (mine > Row<T>::kList - EV) at = list, mine = Row<T>::kList + 1;
      };
      if (use_k) {
        // a vector whose largest logit lies below the bracket is skipped; the bound allows for the
        // roundings of -x
        const float reach = hi / sc.c;
        float floor = mx - reach - (fabsf(mx) + reach) * 9.5367431640625e-7f;
        if (only_max || !(floor > -inf)) floor = -inf;
        walk<1, 4>(row, vb, ve, lane, [&](const uint4 &q, int) {
          if (!(Row<T>::max_of(q) >= floor)) return;
          room();
          float z[EV];
          unpack(q, z);
#pragma unroll
          for (int i = 0; i < EV; ++i)
            if (sc.neg_x(z[i]) < hi) {
              *at = static_cast<T>(z[i]);
              at += kThreads;
              ++mine;
            }
        });
      } else {
        const uint32_t lo_key = __float_as_uint(lo), span = __float_as_uint(hi) - lo_key;
        walk<1, 4>(row, vb, ve, lane, [&](const uint4 &q, int) {
          room();
          float z[EV];
          unpack(q, z);
#pragma unroll
          for (int i = 0; i < EV; i += 2) {
            float nx[2];
            sc.neg_x2(z[i], z[i + 1], nx);
            const uint32_t w[2] = {weight_of(exp2_neg(nx[0])), weight_of(exp2_neg(nx[1]))};
            all += w[0] + w[1];  // (at most 2^31)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (nx[j] < lo) above += w[j];
              if (__float_as_uint(nx[j]) - lo_key < span) {
                *at = static_cast<T>(z[i + j]);
                at += kThreads;
                ++mine;
              }
            }
          }
        });
      }
      uint32_t cnt = static_cast<uint32_t>(mine), over = mine > Row<T>::kList ? 1u : 0u;
      uint64_t ab = above, in_mass = 0;
      if (over) mine = 0;
      else if (!use_k)
        for (int i = 0; i < mine; ++i) in_mass += weight_of(exp2_neg(sc.neg_x(static_cast<float>(list[i * kThreads]))));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        cnt += __shfl_xor_sync(0xFFFFFFFFu, cnt, o);
        over |= __shfl_xor_sync(0xFFFFFFFFu, over, o);
        ab += __shfl_xor_sync(0xFFFFFFFFu, ab, o);
        in_mass += __shfl_xor_sync(0xFFFFFFFFu, in_mass, o);
        all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
      }
      if (lane == 0) {
        red_add_cluster_u32(to_first(&s.bracket_n), cnt);
        if (over) red_add_cluster_u32(to_first(&s.overflow), 1u);
        if (use_p) {
          red_add_cluster_u64(to_first(&s.above), ab);
          red_add_cluster_u64(to_first(&s.bracket_mass), in_mass);
          red_add_cluster_u64(to_first(&s.total), all);
        }
      }
      row_sync(ctas);
      n = first_u32(s.bracket_n);
      listed = first_u32(s.overflow) == 0;
      if (!use_k) {
        total = first_u64(s.total);
        const uint64_t upto = first_u64(s.above);
        const uint64_t target = mass_target(top_p, total);
        // (and min-p must not reach above the bracket, whose mass is not looked at token by token)
        listed = listed && upto < target && target <= upto + first_u64(s.bracket_mass) &&
                 (edge_lo == 0 || exp2_neg(lo) >= min_p);
      }
    }

    // The keys of the bracket, or of the row.
    auto each_key = [&](uint32_t lo, uint32_t hi, auto &&f) {
      if (listed) {
        for (int i = 0; i < mine; ++i) {
          const uint32_t key = __float_as_uint(sc.neg_x(static_cast<float>(list[i * kThreads])));
          if (key >= lo && key < hi) f(key);
        }
      } else {
        walk<1, 1>(row, vb, ve, lane, [&](const uint4 &q, int) {
          float z[EV];
          unpack(q, z);
#pragma unroll
          for (int i = 0; i < EV; ++i) {
            const float nx = sc.neg_x(z[i]);
            const uint32_t key = __float_as_uint(nx);
            if (nx < 32.0f && key >= lo && key < hi) f(key);
          }
        });
      }
    };
    auto add_key = [&](uint32_t *count, uint64_t *mass, uint32_t key) {
      atomicAdd(count, 1u);
      atomicAdd(reinterpret_cast<unsigned long long *>(mass),
                static_cast<unsigned long long>(weight_of(exp2_neg(__uint_as_float(key)))));
    };
    if (!listed) {  // counts and masses of the classes of the whole row
      row_sync(ctas);  // (the first CTA's bins have been read)
      clear_classes();
      row_sync(ctas);
      each_key(0u, kNoCut, [&](uint32_t key) {
        const int b = static_cast<int>(__uint_as_float(key) * 32.0f);
        add_key(&s.count[b], &s.mass[b], key);
      });
      __syncthreads();
      add_to_first(s.count, s.mass, kClasses);
      row_sync(ctas);
    }

    // 4. Keeps the shortest beginning of the order whose count (or mass) reaches target, with then_p also
    // top-p of what that keeps; returns the mass of the first.  Every branch goes by what the first CTA
    // holds, so all CTAs of the row take it alike.
    int level = 0;  // splits made so far: they alternate between two sets of bins
    auto keep = [&](bool by_mass, uint64_t target, int which, bool then_p) -> uint64_t {
      uint32_t lo, hi, left = n;
      if (listed) {
        lo = __float_as_uint(class_edge(edge_lo));
        hi = __float_as_uint(class_edge(edge_hi));
        if (rank == 0) {
          if (threadIdx.x == 0) s.found.count = 0, s.found.mass = s.above;
          __syncthreads();
        }
      } else {
        if (rank == 0) {
          if (threadIdx.x == 0) s.found.count = s.found.mass = 0;
          __syncthreads();
          find_bin(s, s.count, s.mass, kClasses, by_mass, target);
        }
        row_sync(ctas);
        if (!first_u32(s.found.ok)) return 0;  // fewer tokens have weight: nothing to cut
        const uint32_t bin = first_u32(s.found.bin);
        lo = __float_as_uint(class_edge(bin));
        hi = __float_as_uint(class_edge(bin + 1));
        left = first_u32(s.found.n);
      }
      while (left > kFew && hi - lo > 1) {
        const int buf = level++ & 1;
        int shift = 0;
        while (((hi - lo - 1) >> shift) >= kSplit) ++shift;
        each_key(lo, hi, [&](uint32_t key) {
          const uint32_t b = (key - lo) >> shift;
          if (listed) {
            // (a CTA's lists hold at most 2^15 keys: neither half of the weights' sum can overflow)
            const uint32_t w = weight_of(exp2_neg(__uint_as_float(key)));
            atomicAdd(&s.part_count[buf][b], 1u);
            atomicAdd(&s.part_lo[b], w & 0xFFFFu);
            atomicAdd(&s.part_hi[b], w >> 16);
          } else {
            add_key(&s.part_count[buf][b], &s.part_mass[buf][b], key);
          }
        });
        __syncthreads();
        for (int i = threadIdx.x; i < kSplit; i += kThreads) {
          if (listed && s.part_count[buf][i]) {
            // (added, not stored: in the first CTA other CTAs' masses arrive at the same time)
            red_add_cluster_u64(map_to_rank(smem_u32(&s.part_mass[buf][i]), rank),
                                (static_cast<uint64_t>(s.part_hi[i]) << 16) + s.part_lo[i]);
            s.part_lo[i] = s.part_hi[i] = 0;
          }
          // (nobody adds to the other set before the next barrier)
          s.part_count[buf ^ 1][i] = 0, s.part_mass[buf ^ 1][i] = 0;
        }
        __syncthreads();
        add_to_first(s.part_count[buf], s.part_mass[buf], kSplit);
        row_sync(ctas);
        if (rank == 0) find_bin(s, s.part_count[buf], s.part_mass[buf], kSplit, by_mass, target);
        row_sync(ctas);
        lo += first_u32(s.found.bin) << shift;
        hi = min(hi, lo + (1u << shift));
        left = first_u32(s.found.n);
      }
      Cut got;
      uint64_t mass;
      if (hi - lo == 1) {
        const uint64_t w = weight_of(exp2_neg(__uint_as_float(lo))), m0 = first_u64(s.found.mass);
        const uint64_t before = by_mass ? m0 : first_u64(s.found.count), each = by_mass ? w : 1;
        got = Cut{lo, static_cast<uint32_t>((target - before + each - 1) / each)};
        mass = m0 + got.r * w;
      } else {
        each_key(lo, hi, [&](uint32_t key) { s.few[atomicAdd(&s.few_n[which], 1u)].x = key; });
        __syncthreads();
        if (rank != 0) {
          const uint32_t have = s.few_n[which];
          if (threadIdx.x == 0 && have) s.base = atom_add_cluster_u32(to_first(&s.few_n[which]), have);
          __syncthreads();
          for (uint32_t i = threadIdx.x; i < have; i += kThreads) st_cluster_u32(to_first(&s.few[s.base + i].x), s.few[i].x);
        }
        row_sync(ctas);
        if (rank == 0) find_key(s, static_cast<int>(left), by_mass ? 0 : target, target, then_p ? top_p : 1.0f);
        row_sync(ctas);
        got = Cut{first_u32(s.found.key), first_u32(s.found.r)};
        mass = first_u64(s.found.mass);
      }
      row_sync(ctas);  // everyone has read found
      if (got.key < cut.key || (got.key == cut.key && got.r < cut.r)) cut = got;
      return mass;
    };
    // (few keys in the bracket of top-k: both cuts are among them)
    const bool both = use_k && use_p && listed && n <= kFew;
#pragma unroll 1
    for (int which = use_k ? 0 : 1; which < (use_p && !both ? 2 : 1); ++which) {
      if (which == 1 && total == 0) {  // no top-k and no bracket, or fewer than k tokens have weight: the whole row's mass
        if (rank == 0) {
          uint64_t a = 0, b = 0;
          for (int i = threadIdx.x; i < kClasses; i += kThreads) a += s.mass[i];
          const uint64_t own = a;
          block_prefix(s.scan, a, b);
          if (threadIdx.x == kThreads - 1) s.total = a + own;
        }
        row_sync(ctas);
        total = first_u64(s.total);
        row_sync(ctas);
      }
      const uint64_t mass = keep(which == 1, which == 1 ? mass_target(top_p, total) : static_cast<uint64_t>(k), which, both);
      if (which == 0) total = mass;
    }
  }
  // (so a token of the largest weight is always kept, and their total is never zero)
  if (only_first) cut = Cut{0, 1};

  // 5. kept weight and ties, of a key and of a stretch of the row
  uint64_t mass = 0;
  uint32_t ties = 0;
  auto add = [&](uint32_t key) {
    if (key <= cut.key) {
      const float e = exp2_neg(__uint_as_float(key));
      if (e >= min_p) {
        if (key == cut.key) ++ties;
        else mass += weight_of(e);
      }
    }
  };
  auto add_row = [&](int b, int e) {
    walk<1, 2>(row, b, e, lane, [&](const uint4 &q, int) {
      float z[EV];
      unpack(q, z);
#pragma unroll
      for (int i = 0; i < EV; ++i) {
        const float nx = sc.neg_x(z[i]);
        if (nx < 32.0f) add(__float_as_uint(nx));
      }
    });
  };
  // Which of n consecutive stretches holds the target (-1: none); `before` and `left`, the mass before the
  // stretch and the ties still to keep from it on, go by index: ties are kept until r of them are.
  const uint64_t wc = cut.key == kNoCut ? 0 : weight_of(exp2_neg(__uint_as_float(cut.key)));
  uint64_t before = 0, target = 0, total = 0;
  uint32_t left = cut.r;
  auto find = [&](const uint64_t *m, const uint32_t *ti, int n) {
    for (int i = 0; i < n; ++i) {
      const uint32_t kept = min(left, ti[i]);
      const uint64_t held = m[i] + wc * kept;
      if (target < before + held) return i;
      before += held;
      left -= kept;
    }
    return -1;
  };
  // first every warp's piece; then the CTA's warps share the piece that holds the target, and the warp whose
  // part does walks it to the token
  int qb = vb, qe = ve;
#pragma unroll 1
  for (int round = 0;; ++round) {
    mass = 0;
    ties = 0;
    if (round == 0 && listed) {
      // (all that is above the bracket is kept: neither the cut nor min-p reaches there)
      for (int i = 0; i < mine; ++i) add(__float_as_uint(sc.neg_x(static_cast<float>(list[i * kThreads]))));
      mass += above;
    } else {
      add_row(qb, qe);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mass += __shfl_xor_sync(0xFFFFFFFFu, mass, o);
      ties += __shfl_xor_sync(0xFFFFFFFFu, ties, o);
    }
    if (lane == 0) s.warp_mass[warp] = mass, s.warp_ties[warp] = ties;
    __syncthreads();
    if (round == 1) break;
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
    } else {
      if (threadIdx.x == 0) s.cta_mass[0] = cta_mass, s.cta_ties[0] = cta_ties;
      __syncthreads();
    }
    uint32_t all_ties = 0;
    for (int i = 0; i < ctas; ++i) total += s.cta_mass[i], all_ties += s.cta_ties[i];
    total += wc * min(all_ties, cut.r);
    const double want = static_cast<double>(p.uniform[r]) * static_cast<double>(total);
    target = want > 0.0 ? static_cast<uint64_t>(want) : 0;
    if (target >= total) target = total - 1;
    if (find(s.cta_mass, s.cta_ties, ctas) != rank) return;
    const int w0 = find(s.warp_mass, s.warp_ties, kWarps);
    __syncthreads();  // (everyone has read the warps' sums)
    const int pb = piece_at(rank * kWarps + w0), len = piece_at(rank * kWarps + w0 + 1) - pb;
    qb = pb + static_cast<int>(static_cast<int64_t>(warp) * len / kWarps);
    qe = pb + static_cast<int>(static_cast<int64_t>(warp + 1) * len / kWarps);
  }
  if (find(s.warp_mass, s.warp_ties, kWarps) != warp) return;
  for (int v0 = qb; v0 < qe; v0 += 32) {
    float z[EV];
    uint32_t wt[EV];
    uint32_t n_ties = 0;
    const bool in = v0 + lane < qe;
    if (in) unpack(row.load(v0 + lane), z);
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
  st = allow_smem(reinterpret_cast<const void *>(kern), sizeof(Smem), dev.device);
  if (st != NVFP4_OK) return st;
  return check_launch(launch(kern, dim3(static_cast<unsigned>(rows * ctas)), dim3(kThreads), sizeof(Smem), (cudaStream_t)stream,
                             (flags & NVFP4_FLAG_PDL) != 0, ctas, a), name);
}
