"""Gradients of the MoE steps that move rows on the GPU, against the oracle's fp64 loops."""
import numpy as np
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


def bf(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


def routed(seed, tokens, topk, rows, dropped=0.1):
    r = np.random.default_rng(seed)
    pos = r.permutation(rows)[: tokens * topk].reshape(tokens, topk).astype(np.int32)
    pos[r.random(pos.shape) < dropped] = -1
    return pos


CASES = [(1, 1, 8), (1, 8, 2048), (3, 2, 16), (37, 3, 1000), (50, 8, 256), (20, 9, 264), (7, 32, 2056), (300, 8, 512), (5, 4, 7168)]


@pytest.mark.parametrize("tokens,topk,h", CASES)
def test_combine_backward(nv, tokens, topk, h):
    r = np.random.default_rng(h)
    rows = tokens * topk + 5
    pos = routed(tokens, tokens, topk, rows)
    dout, y = bf(r.standard_normal((tokens, h))), bf(r.standard_normal((rows, h)))
    w = torch.from_numpy(r.random((tokens, topk)).astype(np.float32)).cuda()
    dy = torch.full((rows, h), -3.0, dtype=torch.bfloat16, device="cuda")
    _, dw = nv.moe_combine_backward(dout, y, torch.from_numpy(pos).cuda(), w, dy=dy)
    d64, y64 = dout.double().cpu().numpy(), y.double().cpu().numpy()
    want, dots = ofp8.combine_grad(d64, y64, pos, w.double().cpu().numpy())
    named = np.zeros(rows, bool)
    named[pos[pos >= 0]] = True
    got = dy.double().cpu().numpy()
    assert (got[~named] == -3.0).all()
    # an fp32 product (2^-24), one bf16 rounding (2^-8)
    assert (np.abs(got[named] - want[named]) <= np.abs(want[named]) * (2.0 ** -8 + 2.0 ** -23)).all()
    size = np.abs(d64[:, None, :] * np.where(pos[..., None] >= 0, y64[np.maximum(pos, 0)], 0)).sum(2)
    # at most h products and sums of fp32, each rounded once
    assert (np.abs(dw.double().cpu().numpy() - dots) <= (h + 8) * 2.0 ** -24 * size).all()
    assert (dw.cpu().numpy()[pos < 0] == 0).all()
    nv.check_status()


@pytest.mark.parametrize("tokens,topk,h", CASES)
def test_gather_backward(nv, tokens, topk, h):
    r = np.random.default_rng(h + 1)
    rows = tokens * topk + 5
    pos = routed(tokens + 1, tokens, topk, rows)
    pos[0, 0] = -1 if topk == 1 else pos[0, 1]          # the same row twice, or a token with none
    dxs = bf(r.standard_normal((rows, h)))
    dx = nv.moe_gather_backward(dxs, torch.from_numpy(pos).cuda())
    d64 = dxs.double().cpu().numpy()
    want = ofp8.gather_grad(d64, pos)
    size = np.where(pos[..., None] >= 0, np.abs(d64[np.maximum(pos, 0)]), 0).sum(1)
    err = np.abs(dx.double().cpu().numpy() - want)
    assert (err <= np.abs(want) * 2.0 ** -8 + topk * 2.0 ** -23 * size).all()
    nv.check_status()


def test_gradients_of_the_forward_steps_by_differences(nv):
    """The two are the transposes of what moe_gather_rows and moe_combine compute: <dout, J v> = <J^T dout, v>."""
    r = np.random.default_rng(9)
    tokens, topk, h, experts = 40, 4, 64, 6
    ids = torch.from_numpy(np.stack([r.permutation(experts)[:topk] for _ in range(tokens)]).astype(np.int32)).cuda()
    ro, src, pos = nv.moe_sort_by_expert(ids, experts)
    x, y, dout = (bf(r.integers(-4, 5, s)) for s in ((tokens, h), (tokens * topk, h), (tokens, h)))
    w = torch.from_numpy(r.integers(1, 4, (tokens, topk)).astype(np.float32)).cuda()
    # small whole numbers: every product and sum is exact in bf16 or fp32 but for the outputs' rounding
    out = y.double()[pos.long()] * w.double().unsqueeze(2)
    dy, dw = nv.moe_combine_backward(dout, y, pos, w)
    assert float((out.sum(1) * dout.double()).sum()) == float((dy.double() * y.double()).sum()) == float((dw.double() * w.double()).sum())
    xs = nv.moe_gather_rows(x, src)
    dx = nv.moe_gather_backward(y, pos)
    assert float((xs.double() * y.double()).sum()) == float((x.double() * dx.double()).sum())


def test_rows_of_a_wider_buffer_and_bad_rows(nv):
    r = np.random.default_rng(2)
    wide, y = bf(r.standard_normal((30, 80))), bf(r.standard_normal((60, 64)))
    pos, w = torch.from_numpy(routed(3, 30, 2, 60, 0)).cuda(), torch.rand(30, 2, device="cuda")
    dout = wide[:, 8:72]
    want = nv.moe_combine_backward(dout.contiguous(), y, pos, w)
    got = nv.moe_combine_backward(dout, y, pos, w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(nv.NVFP4Error):
        nv.moe_combine_backward(dout, y, pos, w, dy=y)
    one = nv.moe_combine_backward(dout[:1].expand(30, 64), y, pos, w)      # one gradient for every token
    assert torch.equal(one[1], nv.moe_combine_backward(dout[:1].expand(30, 64).contiguous(), y, pos, w)[1])
    nv.check_status()
    bad = pos.clone()
    bad[4, 1] = 60
    dy, dw = nv.moe_combine_backward(dout, y, bad, w)
    assert float(dw[4, 1]) == 0.0
    with pytest.raises(nv.NVFP4Error):
        nv.check_status()
    gone = pos.clone()
    gone[4, 1] = -1
    dx = nv.moe_gather_backward(y, bad)
    assert torch.equal(dx, nv.moe_gather_backward(y, gone))
    with pytest.raises(nv.NVFP4Error):
        nv.check_status()
