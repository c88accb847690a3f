// e4m3 products scaled per block of 128: the dense entry point and its choice of tiles.
#include "fp8_gemm.cuh"

using namespace nvfp4;

namespace {

struct Call {
  const char *name;
  const uint8_t *a, *b;
  int64_t m, n, k;
  int block_b;
  fp8::Args args;
  const DeviceInfo *dev;
  uint32_t flags;
  nvfp4_stream_t stream;
  const float *sfa, *sfb;
};

// Scales of one per row and block: [blocks along K][rows].  One per 128 rows: [blocks of rows][blocks along K].
fp8::Scales row_scales(const float *p, int64_t rows) { return fp8::Scales{p, 0, 1, rows}; }
fp8::Scales block_scales(const float *p, int64_t nk) { return fp8::Scales{p, 0, nk, 1}; }

// CTAs of a cluster that share a tile's K (SWAP): as many as leave no SM without one, at most 8.
int swap_splits(int64_t tiles, int nk, int sms) {
  int64_t s = tiles > 0 ? sms / tiles : 1;
  if (s > 8) s = 8;
  if (s > nk) s = nk;
  return s < 1 ? 1 : static_cast<int>(s);
}

template <class C>
nvfp4_status_t run(const Call &c) {
  fp8::Args args = c.args;
  const fp8::Scales sa = row_scales(c.sfa, c.m);
  const fp8::Scales sb = c.block_b == 128 ? block_scales(c.sfb, args.nk) : row_scales(c.sfb, c.n);
  const int64_t p = C::SWAP ? c.n : c.m, q = C::SWAP ? c.m : c.n;
  args.sp = C::SWAP ? sb : sa;
  args.sq = C::SWAP ? sa : sb;
  args.p_rows = static_cast<int>(p);
  args.q_rows = static_cast<int>(q);
  args.p_tiles = static_cast<int>(ceil_div(p, 128));
  args.q_tiles = static_cast<int>(ceil_div(q, C::NT));
  const int64_t tiles = static_cast<int64_t>(args.p_tiles) * args.q_tiles;
  if (tiles >= (1LL << 31) - 1024) return fail(NVFP4_ERR_INVALID_ARG, "%s: problem too large", c.name);
  args.splits = C::SWAP ? swap_splits(tiles, args.nk, c.dev->sm_count) : 1;
  return fp8::launch_gemm<C>(c.name, C::SWAP ? c.b : c.a, p, C::SWAP ? c.a : c.b, q, c.k, tiles, args, *c.dev, c.flags,
                             c.stream);
}

template <int NT>
nvfp4_status_t run_swap(const Call &c) {
  return c.block_b == 128 ? run<fp8::Cfg<NT, true, false, true, fp8::kDense>>(c)
                          : run<fp8::Cfg<NT, true, true, true, fp8::kDense>>(c);
}
template <int NT>
nvfp4_status_t run_rows(const Call &c) {
  return c.block_b == 128 ? run<fp8::Cfg<NT, false, true, false, fp8::kDense>>(c)
                          : run<fp8::Cfg<NT, false, true, true, fp8::kDense>>(c);
}

// Tiles of more than 128 tokens, by what they cost: rounds of tiles over the SMs times the time of a tile's blocks.
// Measured (ns a block): tokens in the lanes 270, 310 and 460 at 64, 128 and 256 columns with a scale per block of
// B, 310, 440 and 630 with one per row; the weight in the lanes (whose K a cluster can share) 310 and 440 at 64
// and 128 columns, and 2500 ns to join a cluster's parts.
enum Choice { kRows64, kRows128, kRows256, kSwap64, kSwap128 };
Choice choose(int64_t m, int64_t n, int nk, bool per_row, int sms) {
  const int64_t rows_ns[3] = {per_row ? 310 : 270, per_row ? 440 : 310, per_row ? 630 : 460}, swap_ns[2] = {310, 440};
  Choice best = kRows256;
  double least = 1e300;
  for (int i = 0; i < 5; ++i) {
    double cost;
    if (i < 3) {
      const int64_t tiles = ceil_div(m, 128) * ceil_div(n, 64LL << i);
      cost = static_cast<double>(ceil_div(tiles, sms)) * nk * rows_ns[i];
    } else {
      const int64_t tiles = ceil_div(n, 128) * ceil_div(m, 64LL << (i - 3));
      const int s = swap_splits(tiles, nk, sms);
      cost = static_cast<double>(ceil_div(tiles, sms)) * ceil_div(nk, s) * swap_ns[i - 3] + (s > 1 ? 2500 : 0);
    }
    if (cost < least) {
      least = cost;
      best = static_cast<Choice>(i);
    }
  }
  return best;
}

}  // namespace

extern "C" nvfp4_status_t fp8_gemm(const uint8_t *a, const float *sfa, const uint8_t *b, const float *sfb, int block_b,
                                   void *d, int d_type, int accumulate, int64_t m, int64_t n, int64_t k, uint32_t flags,
                                   nvfp4_stream_t stream) {
  clear_error();
  const char *name = "fp8_gemm";
  nvfp4_status_t st = fp8::check_product(name, m, n, k, d_type, accumulate, flags);
  if (st != NVFP4_OK) return st;
  if (block_b != 1 && block_b != 128) return fail(NVFP4_ERR_INVALID_ARG, "%s: block_b=%d (1 or 128)", name, block_b);
  if (m == 0) return NVFP4_OK;
  if (!a || !sfa || !b || !sfb || !d) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(d, 16) || !aligned(sfa, 4) || !aligned(sfb, 4))
    return fail(NVFP4_ERR_MISALIGNED, "%s: a, b and d need 16-B, the scales 4-B alignment", name);
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  Call c{name, a, b, m, n, k, block_b, fp8::Args{}, &dev, flags, stream, sfa, sfb};
  fp8::fill_args(c.args, d, d_type, accumulate, n, k, dev, flags);
  if (m <= 16) return run_swap<16>(c);
  if (m <= 32) return run_swap<32>(c);
  if (m <= 64) return run_swap<64>(c);
  if (m <= 128) return run_swap<128>(c);
  switch (choose(m, n, c.args.nk, block_b == 1, dev.sm_count)) {
    case kRows64: return run_rows<64>(c);
    case kRows128: return run_rows<128>(c);
    case kSwap64: return run_swap<64>(c);
    case kSwap128: return run_swap<128>(c);
    default: return run_rows<256>(c);
  }
}
