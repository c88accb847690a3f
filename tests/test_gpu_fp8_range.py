"""The 8-bit products over the whole range of scales that the quantiser gives (2^-100 / 448 to the largest fp32 / 448):
two scales whose product leaves fp32 still scale a block's sums that stay in it, whatever tiles the sizes choose."""
import pytest
import torch

from oracle import fp8 as ofp8

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_bf16_gb300 as m
    torch.cuda.set_device(0)
    yield m
    m.check_status()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(seed, *shape):
    c = torch.randint(0, 256, shape, generator=gen(seed), device="cuda", dtype=torch.uint8)
    c[(c & 0x7F) == 0x7F] = 0x30
    return c.view(torch.float8_e4m3fn)


def scales(seed, exponent, *shape):
    """Between 2^exponent and twice that."""
    return ((1.0 + torch.rand(*shape, generator=gen(seed), device="cuda").double()) * 2.0 ** exponent).to(F32)


def halves(a, b):
    """`a` keeps the first half of every block of 128, `b` the second: every block's sum is zero."""
    for t, other in ((a, 1), (b, 0)):
        col = torch.arange(t.shape[-1], device="cuda")
        t.view(torch.uint8)[..., (col % 128 // 64) == other] = 0


def rows64(q, s):
    return q.double() * s.double().t().repeat_interleave(128, 1)[:, : q.shape[1]]


def blocks64(q, s):
    n, k = q.shape[-2:]
    return q.double() * s.double().repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]


def within(d, a, b, k):
    """Half a step of D's type, the slack of the sums (see ofp8.product_slack), and the least fp32 number for each block
    added, where the sums are below the normal numbers."""
    r = a @ b.t()
    tol = ofp8.product_slack(k) * (a.abs() @ b.abs().t()) + -(-k // 128) * 2.0 ** -149
    tol = tol + torch.finfo(d.dtype).eps / 2 * (r.abs() + tol)
    err = (d.double() - r).abs()
    bad = ~(err <= tol)                                 # (a NaN is bad)
    assert not bool(bad.any()), (int(bad.sum()), tuple(d.shape), tuple(bad.nonzero()[0].tolist()))


# exponents of the two operands' scales, and whether the sums of the blocks are zero.  A block's sum is between 2^-18 and
# 2^24.7 in magnitude; the results are normal fp32 numbers but for the first pair's smallest.
PAIRS = [(-74, -74, False), (-60, -70, False), (64, 64, True), (119, 119, True), (112, -100, False), (-100, 112, False),
         (118, -108, False), (-108, 118, False), (118, -30, False), (-30, 118, False), (-5, -8, False)]
# up to 128 rows with the weight in the lanes, beyond each kind of tile
GEMMS = [(1, 256, 512), (16, 300, 400), (40, 256, 384), (128, 256, 256), (129, 256, 256), (140, 1000, 256), (300, 1008, 2080),
         (1030, 2040, 256), (2000, 1536, 400), (2100, 4100, 256)]


@pytest.mark.parametrize("block_b", [128, 1])
@pytest.mark.parametrize("ea,eb,zero", PAIRS)
@pytest.mark.parametrize("m,n,k", GEMMS)
def test_gemm(nv, m, n, k, ea, eb, zero, block_b):
    kb = -(-k // 128)
    a, sa, b = codes(m, m, k), scales(1, ea, kb, m), codes(n, n, k)
    sb = scales(2, eb, -(-n // 128), kb) if block_b == 128 else scales(2, eb, kb, n)
    if zero:
        halves(a, b)
    d = nv.fp8_gemm(a, sa, b, sb, block_b=block_b, out_dtype=F32)
    within(d, rows64(a, sa), blocks64(b, sb) if block_b == 128 else rows64(b, sb), k)
    if zero:
        assert bool((d == 0).all())


def test_block_of_a_scale_product_below_fp32(nv):
    """Magnitudes of 3e-20 on both sides: the sums are normal numbers (1.15e-37), the scales' product is not."""
    for m in (128, 129, 2000):
        x = torch.full((m, 128), 3e-20, device="cuda")
        w = torch.full((1536, 128), 3e-20, device="cuda")
        d = nv.fp8_gemm(*nv.fp8_quantize(x), *nv.fp8_quantize_weight(w), out_dtype=F32)
        assert bool(((d.double() - 128 * 9e-40).abs() <= 128 * 9e-40 * 2.0 ** -20).all())     # (3e-20 in fp32, four roundings)


@pytest.mark.parametrize("ea,eb,zero", PAIRS)
@pytest.mark.parametrize("counts,n,k", [([1, 3], 200, 256), ([5, 0, 11], 130, 400), ([16, 15, 1, 30], 256, 256), ([17, 40, 0, 33], 264, 256),
                                        ([300, 700, 0, 50, 1200], 2048, 256)])
def test_grouped(nv, counts, n, k, ea, eb, zero):
    ro = [sum(counts[:i]) for i in range(len(counts) + 1)]
    t, e, kb = ro[-1], len(counts), -(-k // 128)
    a, sa, b, sb = codes(3, t, k), scales(4, ea, kb, t), codes(5, e, n, k), scales(6, eb, e, -(-n // 128), kb)
    if zero:
        halves(a, b)
    d = nv.fp8_grouped_gemm(a, sa, torch.tensor(ro, device="cuda"), b, sb, out_dtype=F32)
    va = rows64(a, sa)
    for i in range(e):
        within(d[ro[i]: ro[i + 1]], va[ro[i]: ro[i + 1]], blocks64(b[i], sb[i]), k)


@pytest.mark.parametrize("ea,eb,zero", PAIRS)
def test_weight_grad(nv, ea, eb, zero):
    counts, n, k, p = [128, 0, 256], 200, 400, 384 + 3 * 128
    a, b = codes(7, n, p), codes(8, k, p)
    sa, sb = scales(9, ea, p // 128, n), scales(10, eb, p // 128, k)
    if zero:
        halves(a, b)
    d = nv.fp8_grouped_weight_grad(a, sa, b, sb, torch.tensor([0, 128, 128, 384], device="cuda"), out_dtype=F32)
    va, vb = rows64(a, sa), rows64(b, sb)
    for i, lo, hi in ((0, 0, 128), (1, 0, 0), (2, 128, 384)):
        within(d[i], va[:, lo:hi], vb[:, lo:hi], max(1, hi - lo))
    assert sum(counts) == 384


@pytest.mark.parametrize("block_b", [128, 1])
@pytest.mark.parametrize("m,n,k", GEMMS)
def test_scales_far_out_leave_the_neighbours_as_they_were(nv, m, n, k, block_b):
    """Rows and columns whose scales are ordinary get the same bits beside others of the far ends of the range."""
    kb = -(-k // 128)
    a, sa, b = codes(m, m, k), scales(1, -5, kb, m), codes(n, n, k)
    sb = scales(2, -8, -(-n // 128), kb) if block_b == 128 else scales(2, -8, kb, n)
    want = nv.fp8_gemm(a, sa, b, sb, block_b=block_b, out_dtype=F32)
    row = torch.arange(m, device="cuda") % 7
    great, least = row == 3, row == 5
    ordinary = ~(great | least)
    far_a, far_b = sa.clone(), sb.clone()
    far_a[:, great] = scales(3, 116, kb, m)[:, great]
    far_a[:, least] = scales(3, -108, kb, m)[:, least]
    got = nv.fp8_gemm(a, far_a, b, sb, block_b=block_b, out_dtype=F32)
    assert torch.equal(got[ordinary], want[ordinary])
    if block_b == 1:
        cols = torch.arange(n, device="cuda") % 5 == 2
        far_b[:, cols] = scales(4, 117, kb, n)[:, cols]
        got = nv.fp8_gemm(a, sa, b, far_b, block_b=1, out_dtype=F32)
        assert torch.equal(got[:, ~cols], want[:, ~cols])
        got = nv.fp8_gemm(a, far_a, b, far_b, block_b=1, out_dtype=F32)     # 2^-108 by 2^117
        within(got[least], rows64(a, far_a)[least], rows64(b, far_b), k)
    else:
        far_a[:, great] = scales(3, -40, kb, m)[:, great]
        far_b[::2] *= 2.0 ** -100                         # by 2^-108: products below fp32's numbers and others beside them
        want, got = (nv.fp8_gemm(a, s, b, far_b, out_dtype=F32) for s in (sa, far_a))
        assert torch.equal(got[ordinary], want[ordinary])
        within(got[~least], rows64(a, far_a)[~least], blocks64(b, far_b), k)
