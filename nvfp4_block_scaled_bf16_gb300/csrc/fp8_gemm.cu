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

// CTAs of a cluster that share a tile's K (SWAP), at most 8 and no more than leave all clusters room at once.  One CTA
// an SM: as many as that.  Two: as few as reach four fifths of the SMs (32 x 4096 x 7168: 4 CTAs a tile 10.4 us, 8
// 12.0; 1 x 14336 x 4096: 1 14.4, 2 12.5).
template <class C>
int splits_of(const Call &c) {
  if (!C::SWAP) return 1;
  const int64_t tiles = ceil_div(c.n, 128) * ceil_div(c.m, C::NT);
  const int sms = c.dev->sm_count;
  if (tiles > sms) return 1;
  int64_t s = C::CTAS == 1 ? sms / tiles : ceil_div(sms * 4LL, 5 * tiles);
  if (s > 8) s = 8;
  if (s > c.args.nk) s = c.args.nk;
  const void *fn = reinterpret_cast<const void *>(fp8::fp8_gemm_kernel<C>);
  if (s > 1 && allow_smem(fn, C::SMEM, c.dev->device) != NVFP4_OK) return 1;
  while (s > 1 && tiles > resident_clusters(fn, C::THREADS, C::SMEM, static_cast<int>(s), c.dev->device)) --s;
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
  args.splits = splits_of<C>(c);
  return fp8::launch_gemm<C>(c.name, C::SWAP ? c.b : c.a, p, C::SWAP ? c.a : c.b, q, c.k, tiles, args, *c.dev, c.flags,
                             c.stream);
}

template <int NT, bool PER_ROW>
using Swap = fp8::Cfg<NT, true, PER_ROW, true, fp8::kDense>;
template <int NT, bool PER_ROW>
using Rows = fp8::Cfg<NT, false, true, PER_ROW, fp8::kDense>;

// Tiles of more than 128 tokens, by what they cost: rounds of tiles over the SMs times the time of a tile's blocks.
// Measured (ns a block): tokens in the lanes 270, 310 and 460 at 64, 128 and 256 columns with a scale per block of
// B, 310, 440 and 630 with one per row; the weight in the lanes (whose K a cluster can share) 310 and 440 at 64
// and 128 columns, 1000 more for a wider tile's ends, and 1400 to join a cluster's parts (all before the test of the
// scales' range, which adds 1 to 5 %).
template <bool PER_ROW>
nvfp4_status_t run_many(const Call &c) {
  const int64_t rows_ns[3] = {PER_ROW ? 310 : 270, PER_ROW ? 440 : 310, PER_ROW ? 630 : 460}, swap_ns[2] = {310, 440};
  const int splits[2] = {splits_of<Swap<64, PER_ROW>>(c), splits_of<Swap<128, PER_ROW>>(c)};
  int best = 2;
  double least = 1e300;
  for (int i = 0; i < 5; ++i) {
    const bool rows = i < 3;
    const int64_t width = 64LL << (rows ? i : i - 3);
    const int64_t tiles = rows ? ceil_div(c.m, 128) * ceil_div(c.n, width) : ceil_div(c.n, 128) * ceil_div(c.m, width);
    const double rounds = static_cast<double>(ceil_div(tiles, c.dev->sm_count));
    double cost = rows ? rounds * c.args.nk * rows_ns[i] : rounds * ceil_div(c.args.nk, splits[i - 3]) * swap_ns[i - 3];
    if (!rows) cost += (splits[i - 3] > 1 ? 1400 : 0) + (i == 4 ? 1000 : 0);
    if (cost < least) {
      least = cost;
      best = i;
    }
  }
  switch (best) {
    case 0: return run<Rows<64, PER_ROW>>(c);
    case 1: return run<Rows<128, PER_ROW>>(c);
    case 2: return run<Rows<256, PER_ROW>>(c);
    case 3: return run<Swap<64, PER_ROW>>(c);
    default: return run<Swap<128, PER_ROW>>(c);
  }
}

// Up to 128 tokens: the weight in the lanes, the narrowest tile that holds them.
template <bool PER_ROW>
nvfp4_status_t run_any(const Call &c) {
  if (c.m <= 16) return run<Swap<16, PER_ROW>>(c);
  if (c.m <= 32) return run<Swap<32, PER_ROW>>(c);
  if (c.m <= 64) return run<Swap<64, PER_ROW>>(c);
  if (c.m <= 128) return run<Swap<128, PER_ROW>>(c);
  return run_many<PER_ROW>(c);
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
  return block_b == 128 ? run_any<false>(c) : run_any<true>(c);
}
