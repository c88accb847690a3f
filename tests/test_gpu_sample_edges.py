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
