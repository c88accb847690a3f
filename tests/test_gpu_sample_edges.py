"""The draw of a token at the edges of its arguments: every row is written, whatever the filters say."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_bf16_gb300 as m
    return m


def vec(v, rows, dtype=torch.float32):
    return None if v is None else torch.full((rows,), v, dtype=dtype, device="cuda")


def draw(nv, z, u, t=None, k=None, p=None, mp=None):
    """The draw into outputs that hold values no draw gives, so that a row left out shows."""
    rows = z.shape[0]
    tok = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((rows,), NAN, device="cuda")
    nv.sample_tokens(z, torch.tensor(u, dtype=torch.float32, device="cuda"), vec(t, rows), vec(k, rows, torch.int32),
                     vec(p, rows), vec(mp, rows), tokens=tok, logprobs=lp)
    return tok.cpu().numpy(), lp.cpu().numpy()


# one CTA a row, eight, and rows enough for two
@pytest.mark.parametrize("rows,v", [(2, 7), (2, 1000), (2, 40000), (100, 40000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("min_p", [1.5, float("inf"), NAN])
@pytest.mark.parametrize("kw", [dict(), dict(k=5), dict(p=0.9), dict(k=5, p=0.9), dict(k=1 << 20), dict(t=0.7, p=0.0)])
def test_min_p_that_nothing_passes_keeps_the_first_token(nv, rows, v, dtype, min_p, kw):
    """The first token of the order stays: the largest logit, the lowest index of those that share it."""
    z = torch.randn(rows, v, generator=torch.Generator().manual_seed(v)).to(dtype)
    z[:, v // 2] = z[:, v - 1] = 9.0
    u = np.linspace(0.0, 0.999, rows).tolist()
    tok, lp = draw(nv, z.cuda(), u, mp=min_p, **kw)
    assert (tok == v // 2).all() and (lp == 0.0).all()


# Row positions that one thread meets one after the other, when eight CTAs share an aligned row: the first vector
# of 16 bytes of a warp's piece and the one 32 vectors on.
def later(dtype):
    return 32 * (4 if dtype == torch.float32 else 8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rest", [-1.0, -40.0])
@pytest.mark.parametrize("kw,n", [(dict(), 0), (dict(k=2), 2), (dict(p=1e-6), 1), (dict(k=2, p=0.75), 2), (dict(k=40), 0),
                                  (dict(mp=0.5), 2), (dict(t=0.0), 1), (dict(k=2, mp=0.5, p=0.9), 2)])
def test_the_two_zeros_are_one_logit(nv, dtype, rest, kw, n):
    """-0 and then +0 as a row's largest logits weigh the same and tie by index; n: how many of them are kept alone."""
    v = 64000
    z = torch.full((2, v), rest, dtype=dtype, device="cuda")
    z[:, 0], z[:, later(dtype)] = -0.0, 0.0
    u = [0.25, 0.75]
    tok, lp = draw(nv, z, u, **kw)
    same = draw(nv, z + 0.0, u, **kw)          # every zero positive
    assert np.array_equal(tok, same[0]) and np.array_equal(lp, same[1])
    if n:
        assert tok.tolist() == [0, later(dtype) if n == 2 else 0]
        assert np.abs(lp + np.log(n)).max() < 1e-6


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kw", [dict(k=3), dict(k=700), dict(k=1500), dict(p=0.01), dict(p=0.3), dict(k=900, p=0.5), dict(mp=1.0)])
def test_many_zeros_of_both_signs(nv, dtype, kw):
    """More zeros than keys are compared with one another, as the largest logits of an ordinary row."""
    g = torch.Generator().manual_seed(8)
    for v in (1000, 64000):
        z = -torch.rand(3, v, generator=g).to(dtype) * 4.0
        at = torch.randperm(v, generator=g)[: v // 4]
        z[:, at] = 0.0
        z[:, at[::2]] = -0.0
        z = z.cuda()
        u = [0.05, 0.5, 0.95]
        a, b = draw(nv, z, u, **kw), draw(nv, z + 0.0, u, **kw)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
        assert not torch.signbit(z + 0.0)[z == 0].any()
        if kw.get("k", 1000) <= v // 4 and len(kw) == 1 and ("k" in kw or "mp" in kw):
            zeros = np.sort(at.numpy())
            kept = zeros[: kw["k"]] if "k" in kw else zeros
            assert a[0].tolist() == [int(kept[int(np.float64(np.float32(x)) * len(kept))]) for x in u]
