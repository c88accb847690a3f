// e4m3 products scaled per block of 128, expert by expert: the rows' products with their expert's weight, and
// the weights' gradients.
#include "fp8_gemm.cuh"

using namespace nvfp4;

namespace {

template <class C>
nvfp4_status_t grouped(const char *name, const uint8_t *a, const float *sfa, const uint8_t *b, const float *sfb,
                       fp8::Args args, int64_t t, int64_t n, int64_t k, int experts, const DeviceInfo &dev, uint32_t flags,
                       nvfp4_stream_t stream) {
  const int64_t nb = ceil_div(n, 128);
  const fp8::Scales sa{sfa, 0, 1, t}, sb{sfb, nb * args.nk, args.nk, 1};
  args.sp = C::SWAP ? sb : sa;
  args.sq = C::SWAP ? sa : sb;
  args.p_rows = args.q_rows = static_cast<int>(n);
  args.p_tiles = static_cast<int>(ceil_div(n, 128));
  args.q_tiles = static_cast<int>(ceil_div(n, C::NT));
  args.splits = 1;
  // sum over experts of ceil(rows / tile) <= min(rows, ceil(t / tile) + experts)
  const int64_t tt = C::SWAP ? C::NT : 128;
  int64_t bound = ceil_div(t, tt) + experts;
  if (bound > t) bound = t;
  bound *= C::SWAP ? args.p_tiles : args.q_tiles;
  if (bound >= (1LL << 31) - 1024) return fail(NVFP4_ERR_INVALID_ARG, "%s: problem too large", name);
  const int64_t br = n * experts;
  return fp8::launch_gemm<C>(name, C::SWAP ? b : a, C::SWAP ? br : t, C::SWAP ? a : b, C::SWAP ? t : br, k, bound, args, dev,
                             flags, stream);
}

template <int NT>
using Swapped = fp8::Cfg<NT, true, false, true, fp8::kGrouped>;
template <int NT>
using Rows = fp8::Cfg<NT, false, true, false, fp8::kGrouped>;
using Grad = fp8::Cfg<256, false, true, true, fp8::kWgrad>;

nvfp4_status_t check_experts(const char *name, int experts, int64_t n) {
  if (experts < 1 || experts > fp8::kMaxExperts)
    return fail(NVFP4_ERR_INVALID_ARG, "%s: num_experts=%d (1..%d)", name, experts, fp8::kMaxExperts);
  if (n * experts >= (1LL << 31)) return fail(NVFP4_ERR_INVALID_ARG, "%s: experts * n too large", name);
  return NVFP4_OK;
}

}  // namespace

extern "C" nvfp4_status_t fp8_grouped_gemm(const uint8_t *a, const float *sfa, const int64_t *row_offsets, int num_experts,
                                           const uint8_t *b, const float *sfb, void *d, int d_type, int64_t t, int64_t n,
                                           int64_t k, uint32_t flags, nvfp4_stream_t stream) {
  clear_error();
  const char *name = "fp8_grouped_gemm";
  nvfp4_status_t st = fp8::check_product(name, t, n, k, d_type, 0, flags);
  if (st == NVFP4_OK) st = check_experts(name, num_experts, n);
  if (st != NVFP4_OK) return st;
  if (t == 0) return NVFP4_OK;
  if (!a || !sfa || !row_offsets || !b || !sfb || !d) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(d, 16) || !aligned(sfa, 4) || !aligned(sfb, 4) ||
      !aligned(row_offsets, 8))
    return fail(NVFP4_ERR_MISALIGNED, "%s: a, b and d need 16-B, row_offsets 8-B, the scales 4-B alignment", name);
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  fp8::Args args{};
  fp8::fill_args(args, d, d_type, 0, n, k, dev, flags);
  args.row_offsets = row_offsets;
  args.experts = num_experts;
  args.total_rows = t;
  // Few rows to an expert: the weight in the lanes and a narrow tile of tokens, for the weight is read from memory
  // once whatever the tile (128 experts of 1536 x 2048, us: 2 rows to an expert 55, 8 rows 68, 16 rows 71; at 48 rows
  // 64 columns of tokens took 87, the rows in the lanes 76, 77 now).  Else the rows in the lanes, 256 columns of the weight to
  // a tile, or 128 where so few tiles would leave SMs idle.
  const int64_t mean = ceil_div(t, num_experts);
  if (mean <= 8)
    return grouped<Swapped<16>>(name, a, sfa, b, sfb, args, t, n, k, num_experts, dev, flags, stream);
  if (mean <= 16)
    return grouped<Swapped<32>>(name, a, sfa, b, sfb, args, t, n, k, num_experts, dev, flags, stream);
  if ((ceil_div(t, 128) + num_experts / 2) * ceil_div(n, 256) < dev.sm_count)
    return grouped<Rows<128>>(name, a, sfa, b, sfb, args, t, n, k, num_experts, dev, flags, stream);
  return grouped<Rows<256>>(name, a, sfa, b, sfb, args, t, n, k, num_experts, dev, flags, stream);
}

extern "C" nvfp4_status_t fp8_grouped_weight_grad(const uint8_t *a, const float *sfa, const uint8_t *b, const float *sfb,
                                                  const int64_t *row_offsets, int num_experts, void *d, int d_type,
                                                  int accumulate, int64_t padded_rows, int64_t n, int64_t k,
                                                  uint32_t flags, nvfp4_stream_t stream) {
  clear_error();
  const char *name = "fp8_grouped_weight_grad";
  if (padded_rows < 128 || padded_rows % 128)
    return fail(NVFP4_ERR_INVALID_ARG, "%s: padded_rows=%lld (a positive multiple of 128)", name, (long long)padded_rows);
  // the products sum over the rows; n and k are the result's sides
  nvfp4_status_t st = fp8::check_product(name, n, k, padded_rows, d_type, accumulate, flags);
  if (st == NVFP4_OK) st = check_experts(name, num_experts, n);
  if (st != NVFP4_OK) return st;
  if (n == 0) return NVFP4_OK;
  if (!a || !sfa || !b || !sfb || !row_offsets || !d)
    return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(d, 16) || !aligned(sfa, 4) || !aligned(sfb, 4) ||
      !aligned(row_offsets, 8))
    return fail(NVFP4_ERR_MISALIGNED, "%s: a, b and d need 16-B, row_offsets 8-B, the scales 4-B alignment", name);
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  fp8::Args args{};
  fp8::fill_args(args, d, d_type, accumulate, k, padded_rows, dev, flags);
  args.sp = fp8::Scales{sfa, 0, 1, n};
  args.sq = fp8::Scales{sfb, 0, 1, k};
  args.p_rows = static_cast<int>(n);
  args.q_rows = static_cast<int>(k);
  args.p_tiles = static_cast<int>(ceil_div(n, 128));
  args.q_tiles = static_cast<int>(ceil_div(k, Grad::NT));
  args.d_expert = n * k;
  args.row_offsets = row_offsets;
  args.experts = num_experts;
  args.total_rows = padded_rows;
  const int64_t tiles = static_cast<int64_t>(args.p_tiles) * args.q_tiles * num_experts;
  if (tiles >= (1LL << 31) - 1024) return fail(NVFP4_ERR_INVALID_ARG, "%s: problem too large", name);
  return fp8::launch_gemm<Grad>(name, a, n, b, k, padded_rows, tiles, args, dev, flags, stream);
}
