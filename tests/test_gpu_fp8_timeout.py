"""A wait that runs out in every kind of 8-bit product: the copy of the first stage is left out, the bounded waits give up,
the status says so, and the next call gives the right product."""
import pytest
import torch

from oracle import fp8 as ofp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_bf16_gb300 as m
    torch.cuda.set_device(0)
    yield m
    m.check_status()


def codes(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    c[(c & 0x7F) == 0x7F] = 0x30
    return c.view(torch.float8_e4m3fn)


def scales(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.exp(torch.randn(*shape, generator=g, device="cuda"))


def rows64(q, s):
    return q.double() * s.double().t().repeat_interleave(128, 1)[:, : q.shape[1]]


def blocks64(q, s):
    n, k = q.shape[-2:]
    return q.double() * s.double().repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]


def within(d, a, b, k):
    """Half a step of D's type and the slack of the sums (see ofp8.product_slack)."""
    r = a @ b.t()
    tol = ofp8.product_slack(k) * (a.abs() @ b.abs().t())
    tol = tol + torch.finfo(d.dtype).eps / 2 * (r.abs() + tol)
    assert bool(((d.double() - r).abs() <= tol).all())


def gives_up_then_works(nv, call):
    call(nv.FLAG_DEBUG_TIMEOUT | nv.FLAG_DEBUG_SKIP_FIRST_LOAD)
    with pytest.raises(nv.NVFP4Error) as e:
        nv.check_status()
    assert e.value.code == 6
    d = call(0)
    nv.check_status()
    return d


# the weight in the lanes, and tiles of 64, 128 and 256 columns with the tokens in them (the last with 16 scaling warps and
# results that leave as bulk copies)
@pytest.mark.parametrize("block_b", [128, 1])
@pytest.mark.parametrize("m,n,k", [(40, 256, 384), (128, 256, 512), (300, 1008, 2080), (1030, 2040, 256), (2000, 1536, 640)])
def test_gemm(nv, m, n, k, block_b):
    kb = -(-k // 128)
    a, sa, b = codes(1, m, k), scales(2, kb, m), codes(3, n, k)
    sb = scales(4, -(-n // 128), kb) if block_b == 128 else scales(4, kb, n)
    d = gives_up_then_works(nv, lambda flags: nv.fp8_gemm(a, sa, b, sb, block_b=block_b, flags=flags))
    within(d, rows64(a, sa), blocks64(b, sb) if block_b == 128 else rows64(b, sb), k)


# means of up to 8 and 16 rows (the weight in the lanes), few tiles, many
@pytest.mark.parametrize("counts,n,k", [([5, 0, 3], 200, 512), ([16, 12, 1], 256, 640), ([100, 60], 264, 384), ([300, 700, 0, 50, 1200], 2048, 640)])
def test_grouped(nv, counts, n, k):
    ro = [sum(counts[:i]) for i in range(len(counts) + 1)]
    t, e, kb = ro[-1], len(counts), -(-k // 128)
    a, sa, b, sb = codes(5, t, k), scales(6, kb, t), codes(7, e, n, k), scales(8, e, -(-n // 128), kb)
    off = torch.tensor(ro, device="cuda")
    d = gives_up_then_works(nv, lambda flags: nv.fp8_grouped_gemm(a, sa, off, b, sb, flags=flags))
    for i in range(e):
        within(d[ro[i]: ro[i + 1]], rows64(a, sa)[ro[i]: ro[i + 1]], blocks64(b[i], sb[i]), k)


def test_weight_grad(nv):
    n, k, p = 200, 400, 896
    a, b, sa, sb = codes(9, n, p), codes(10, k, p), scales(11, p // 128, n), scales(12, p // 128, k)
    off = torch.tensor([0, 128, 128, 640], device="cuda")
    d = gives_up_then_works(nv, lambda flags: nv.fp8_grouped_weight_grad(a, sa, b, sb, off, flags=flags))
    va, vb = rows64(a, sa), rows64(b, sb)
    for i, (lo, hi) in enumerate(((0, 128), (0, 0), (128, 640))):
        within(d[i], va[:, lo:hi], vb[:, lo:hi], max(1, hi - lo))
