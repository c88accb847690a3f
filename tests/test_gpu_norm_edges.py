"""Norms around a block where an operand is absent, does not matter, or is not finite, by both kernels: rows
go straight to registers (few rows) or are copied ahead (from 4 rows an SM on)."""
import numpy as np
import pytest
import torch

import test_gpu_block_norm as common
from oracle import block

pytestmark = pytest.mark.gpu

BF16, FP32 = 2.0 ** -8, 2.0 ** -17      # as test_gpu_block_norm derives them
ROWS = [(5, 1032), (609, 520), (700, 1032), (620, 4104), (608, 8192), (5, 333), (700, 333)]


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_bf16_gb300 as m
    return m


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def inputs(m, n, stream, gate, seed=0):
    g = torch.Generator().manual_seed(seed + m + n)
    rows = lambda dtype, std: (torch.randn(m, n, generator=g) * std).to(dtype).cuda()  # noqa: E731
    vec = lambda std, mean: (mean + torch.randn(n, generator=g) * std).to(torch.bfloat16).cuda()  # noqa: E731
    return dict(x=rows(stream, 1.0), y=rows(torch.bfloat16, 0.7), dr=rows(stream, 0.1), dh=rows(torch.bfloat16, 0.1),
                w_post=vec(0.2, 1.0), w_pre=vec(0.2, 1.0),
                gate={"none": None, "channel": vec(0.5, 0.0), "token": rows(torch.bfloat16, 0.5)}[gate])


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("m,n", ROWS)
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_backward_without_the_second_norm(nv, m, n, gate, stream, eps):
    """Without dh the stream has no part in any gradient: dx is dx_out, and dy, dw_post and dgate follow the
    formulas with eps = 0 too and whatever the stream holds."""
    d = inputs(m, n, stream, gate)
    kw = dict(y=d["y"], w_post=d["w_post"], gate=d["gate"], residual_scale=0.9, eps=eps)
    dx, dy, dw_pre, dw_post, dgate = nv.block_norm_backward(None, d["dr"], d["x"], None, **kw)
    assert dw_pre is None and torch.equal(dx, d["dr"])
    _, ry, _, rw, rg = block.block_norm_backward(None, f64(d["dr"]), f64(d["x"]), None, f64(d["y"]), f64(d["w_post"]),
                                                 f64(d["gate"]), 0.9, eps, 0.0)
    # magnitudes that enter the results, with the sums of magnitudes in place of the sums
    y, w, b = np.abs(f64(d["y"])), np.abs(f64(d["w_post"])), 0.9 * np.abs(f64(d["dr"]))
    rstd = 1.0 / np.sqrt(np.mean(y * y, axis=1, keepdims=True) + eps)
    yn = y * rstd
    terms = {"dgate": b * yn * w}
    if d["gate"] is not None:
        b = b * np.abs(f64(d["gate"]))
    terms["dy"] = rstd * (b * w + yn * np.mean(b * w * yn, axis=1, keepdims=True))
    terms["dw_post"] = np.sum(b * yn, axis=0)
    if gate == "channel":
        terms["dgate"] = terms["dgate"].sum(axis=0)
    for name, got, ref in (("dy", dy, ry), ("dw_post", dw_post, rw), ("dgate", dgate, rg)):
        assert (got is None) == (ref is None)
        if got is not None:
            rounding = BF16 if got.dtype == torch.bfloat16 else 2.0 ** -23
            assert np.all(np.abs(f64(got) - ref) <= rounding * np.abs(ref) + 2 * FP32 * terms[name] + 1e-30), name
    x = d["x"].clone()
    x[0, 3], x[m // 2, n // 2], x[m - 1, n - 1] = float("nan"), float("inf"), float("-inf")
    for a, c in zip(nv.block_norm_backward(None, d["dr"], x, None, **kw), (dx, dy, None, dw_post, dgate)):
        assert (a is None and c is None) or torch.equal(a, c)


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n", ROWS)
def test_forward_without_the_second_norm(nv, m, n, stream):
    """x_out is the same whether h is asked for or not, in place too."""
    for gate in ("none", "channel", "token"):
        d = inputs(m, n, stream, gate)
        kw = dict(y=d["y"], w_post=d["w_post"], gate=d["gate"], residual_scale=0.7)
        want, _ = nv.block_norm(d["x"], d["w_pre"], **kw)
        got, none = nv.block_norm(d["x"], None, **kw)
        assert none is None and torch.equal(got, want)
        x = d["x"].clone()
        nv.block_norm(x, None, x_out=x, **kw)
        assert torch.equal(x, want)


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("m,n", ROWS)
def test_backward_without_the_norm_after_the_block(nv, m, n, gate, stream):
    """Without w_post y is a factor of dgate alone: dx and dy do not depend on it, finite or not."""
    d = inputs(m, n, stream, gate)
    kw = dict(gate=d["gate"], residual_scale=0.9)
    want = nv.block_norm_backward(d["dh"], d["dr"], d["x"], d["w_pre"], y=d["y"], **kw)
    y = d["y"].clone()
    at = [(0, 3), (m // 2, n // 2), (m - 1, n - 1)]
    for (r, c), v in zip(at, ("nan", "inf", "-inf")):
        y[r, c] = float(v)
    got = nv.block_norm_backward(d["dh"], d["dr"], d["x"], d["w_pre"], y=y, **kw)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b)
    if gate == "token":
        same = torch.ones_like(got[4], dtype=torch.bool)
        for r, c in at:
            same[r, c] = False
        assert torch.equal(got[4][same], want[4][same]) and not torch.isfinite(got[4][~same].float()).any()


@pytest.mark.parametrize("m,n", [(620, 7168), (609, 7040), (608, 8192), (610, 8152)])
def test_rows_too_wide_to_be_copied_ahead(nv, m, n):
    """An fp32 stream with a gate per token: at 7040 to 7168 channels forward and from 8152 on backward two rows do not
    fit beside each other, and the plain kernels take many rows too."""
    d = common.inputs(m, n, torch.float32, True, "token")
    kw = dict(y=d["y"], w_post=d["w_post"], gate=d["gate"], residual_scale=0.7)
    x_out, h = nv.block_norm(d["x"], d["w_pre"], eps=common.EPS, **kw)
    r_ref, h_ref = block.block_norm(f64(d["x"]), f64(d["w_pre"]), f64(d["y"]), f64(d["w_post"]), f64(d["gate"]), 0.7, common.EPS)
    tr, th = common.forward_terms(d, 0.7, 0.0)
    common.check(x_out, r_ref, 2.0 ** -23, tr, "x_out")
    common.check(h, h_ref, BF16, th, "h")
    if n % 16 == 0:
        gs = (2688.0 / h.float().abs().max()).reshape(1)
        q_ref, sf_ref = nv.nvfp4_quantize(h, gs)
        x2, q, sf = nv.block_norm_quantize(d["x"], d["w_pre"], gs, eps=common.EPS, **kw)
        assert torch.equal(x2, x_out) and torch.equal(q, q_ref) and torch.equal(sf, sf_ref)
    common.check_backward(nv, d, 0.7, 0.0)
