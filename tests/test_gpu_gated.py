"""The gated product of a feed-forward block and its backward pass on the GPU against the fp64 forms of
oracle/block.py, over every kind of plan.

Bounds, fixed by the arithmetic.  Each product's fp32 sum is within 1e-5 of its sum of magnitudes S, the
bound the plain product is held to; h = act(g) u then moves by at most 1.13 |u| 1e-5 Sg + |act(g)| 1e-5 Su
(|act'| <= 1.13 for both activations), the gradients by |dh| (|u| 1e-5 Sg + 1.13 * 1e-5 Su) (|act''| <= 1)
and |dh| 1.13 * 1e-5 Sg.  The approximate exponential and reciprocal are within a few fp32 ulps: 2^-19 of
the value, and 2^-19 |dh u| (1 + |g|) where act' cancels.  One rounding to bf16: 2^-8 of the value."""
import numpy as np
import pytest
import torch

from cases import dev, nvfp4_operands
from oracle import block
from oracle import gemm as ogemm

pytestmark = pytest.mark.gpu

ACC, FN, BF16 = 1e-5, 2.0 ** -19, 2.0 ** -8


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_bf16_gb300 as m
    return m


def operands(m, inter, k, seed=0):
    """Operands as nvfp4_gemm's (the weight's rows are the interleaved ones) and the fp64 products."""
    ops = nvfp4_operands(m, 2 * inter, k, seed)
    A = ogemm.dequantize(ops["qa"], ops["sfa"], m, k, 16, "e4m3")
    B = ogemm.dequantize(ops["qb"], ops["sfb"], 2 * inter, k, 16, "e4m3")
    # two factors, so that mixing them up shows
    alpha = np.array([2.0, 0.75], dtype=np.float32) * np.float32(ops["alpha"])
    args = (dev(ops["qa"]), dev(ops["sfa"]), dev(ops["qb"]), dev(ops["sfb"]), torch.from_numpy(alpha).cuda())
    sg, su = block.split_gate_up(np.abs(A) @ np.abs(B).T)
    g, u = block.split_gate_up(A @ B.T)
    a0, a1 = float(alpha[0]), float(alpha[1])
    return args, a0 * g, a1 * u, a0 * sg, a1 * su


def close(got, ref, tol, what):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside, worst {np.max(np.abs(got - ref) / tol):.3g}"


def bounds(g, u, sg, su, kind, dh=None):
    f, df = block.activation(g, kind)
    h = f * u
    out = {"h": (h, BF16 * np.abs(h) + ACC * (1.13 * np.abs(u) * sg + np.abs(f) * su) + FN * np.abs(h) + 1e-30)}
    if dh is not None:
        dg, du = dh * u * df, dh * f
        tg = BF16 * np.abs(dg) + np.abs(dh) * (ACC * (np.abs(u) * sg + 1.13 * su) + FN * np.abs(u) * (1 + np.abs(g))) + 1e-30
        tu = BF16 * np.abs(du) + np.abs(dh) * (ACC * 1.13 * sg + FN * np.abs(f)) + 1e-30
        out["dgu"] = (block.join_gate_up(dg, du), block.join_gate_up(tg, tu))
    return out


# (m, inter, k): what the selector makes of n = 2 inter
PLANS = [
    (1, 16, 32), (1, 48, 96), (3, 16, 4096),                       # smallest
    (1, 2048, 7168), (15, 512, 1024), (16, 512, 1024), (17, 784, 2080), (32, 2048, 1792),  # 32-wide, read and pushed slices
    (9, 64, 512), (31, 96, 1536),                                  # few tiles, long splits
    (33, 512, 1024), (64, 784, 2080), (50, 16, 2048),              # 64-wide
    (100, 784, 2080), (128, 512, 4096), (65, 10240, 256),          # 128-wide, split and whole
    (200, 784, 2080), (256, 512, 4096), (129, 10256, 288),         # 256-wide
    (40, 10240, 320), (5, 20480, 256),                             # more weight tiles than SMs: no split
    (64, 2304, 768),                                               # short K: whole 128 x 128 tiles
    (300, 6528, 512), (257, 8192, 544), (640, 10240, 256),         # CTA pairs, one and two K steps a stage
    (1000, 528, 1056), (640, 512, 2048),                           # 128 x 128 tiles, ragged
    (300, 512, 16384),                                             # stream-K
]


@pytest.mark.parametrize("m,inter,k", PLANS)
def test_forward_and_backward(nv, m, inter, k):
    args, g, u, sg, su = operands(m, inter, k)
    gen = torch.Generator().manual_seed(m + inter + k)
    dh = torch.randn(m, inter, generator=gen).to(torch.bfloat16).cuda()
    for kind in ("silu", "gelu_tanh"):
        want = bounds(g, u, sg, su, kind, dh.double().cpu().numpy())
        h = nv.nvfp4_gated_gemm(*args, activation=kind)
        nv.check_status()
        close(h, *want["h"], f"{kind} h")
        dgu, h2 = nv.nvfp4_gated_gemm_backward(*args, dh, activation=kind)
        nv.check_status()
        close(dgu, *want["dgu"], f"{kind} dgu")
        assert torch.equal(h, h2)


def test_the_plans_are_all_there(nv):
    kinds = set()
    for m, inter, k in PLANS:
        p = nv.nvfp4_gemm_plan(m, 2 * inter, k)
        form = "stream-K" if p["sk_tiles"] else "pair" if p["tile_m"] == 256 else "swap" if p["swap_ab"] else "whole"
        kinds.add((form, p["tile_n"], p["splits"] > 1, form == "pair" and k % 256 == 0))
    for want in (("swap", 32, True, False), ("swap", 32, False, False), ("swap", 64, True, False), ("swap", 64, False, False),
                 ("swap", 128, True, False), ("swap", 256, True, False), ("whole", 128, False, False),
                 ("pair", 256, False, True), ("pair", 256, False, False), ("stream-K", 128, False, False)):
        assert want in kinds, (want, sorted(kinds))


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gradients_against_differences(nv, kind):
    """Gradients along the direction of each product against central differences of the fp64 forward
    pass: scaling a product by 1 + e changes sum(dh h) by e * sum(gradient * product).  The bf16
    gradients are off by 2^-8 of each term, everything before their rounding by far less (2^-8 more
    covers it); the differences, with step 1e-6, by 1e-6 of the terms."""
    m, inter, k = 24, 256, 512
    args, g, u, _, _ = operands(m, inter, k, seed=4)
    dh = torch.randn(m, inter, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    d = dh.double().cpu().numpy()
    dgu, _ = nv.nvfp4_gated_gemm_backward(*args, dh, activation=kind)
    dg, du = block.split_gate_up(dgu.double().cpu().numpy())

    def loss(a, b):
        return np.sum(d * block.activation(a * g, kind)[0] * (b * u))

    e = 1e-6
    for grad, product, want in ((dg, g, (loss(1 + e, 1) - loss(1 - e, 1)) / (2 * e)),
                                (du, u, (loss(1, 1 + e) - loss(1, 1 - e)) / (2 * e))):
        assert abs(np.sum(grad * product) - want) <= (2 * BF16 + 1e-6) * np.sum(np.abs(grad * product))


def test_interleaved_weight_of_two_matrices(nv):
    """From two bf16 weights as a model stores them, through the library's quantiser.  The plain product
    of the same weight gives both pre-activations rounded to bf16: 2^-8 of each."""
    m, inter, k = 8, 160, 256
    gen = torch.Generator().manual_seed(0)
    wg = (torch.randn(inter, k, generator=gen) * 0.05).to(torch.bfloat16).cuda()
    wu = (torch.randn(inter, k, generator=gen) * 0.05).to(torch.bfloat16).cuda()
    x = torch.randn(m, k, generator=gen).to(torch.bfloat16).cuda()
    w = nv.interleave_gate_up(wg, wu)
    assert torch.equal(w[0:16], wg[0:16]) and torch.equal(w[16:32], wu[0:16]) and torch.equal(w[32:48], wg[16:32])
    gsw, gsx = (2688.0 / w.float().abs().max()).reshape(1), (2688.0 / x.float().abs().max()).reshape(1)
    b, sfb = nv.nvfp4_quantize(w, gsw)
    a, sfa = nv.nvfp4_quantize(x, gsx)
    alpha = (1.0 / (gsw * gsx)).repeat(2)
    h = nv.nvfp4_gated_gemm(a, sfa, b, sfb, alpha)
    c = nv.nvfp4_gemm(a, sfa, b, sfb, alpha[:1].contiguous()).double().cpu().numpy()
    g, u = block.split_gate_up(c)
    ref = block.activation(g, "silu")[0] * u
    close(h, ref, 2 * BF16 * (np.abs(ref) + 1.13 * np.abs(g * u)) + 1e-6, "h")


def test_flags_streams_and_empty_batches(nv):
    m, inter, k = 40, 512, 1024
    args, *_ = operands(m, inter, k)
    want = nv.nvfp4_gated_gemm(*args)
    assert torch.equal(want, nv.nvfp4_gated_gemm(*args, flags=nv.FLAG_PDL))
    sm103 = list(args)
    sm103[1] = nv.sf_convert_layout(args[1], m, k // 16)
    sm103[3] = nv.sf_convert_layout(args[3], 2 * inter, k // 16)
    assert torch.equal(want, nv.nvfp4_gated_gemm(*sm103, flags=nv.FLAG_SF_SM103))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h = torch.empty_like(want)
    nv.nvfp4_gated_gemm(*args, h=h, stream=s)
    s.synchronize()
    assert torch.equal(h, want)
    empty = (args[0][:0],) + args[1:]
    assert nv.nvfp4_gated_gemm(*empty).shape == (0, inter)
    dgu, h0 = nv.nvfp4_gated_gemm_backward(*empty, torch.empty(0, inter, dtype=torch.bfloat16, device="cuda"))
    assert dgu.shape == (0, 2 * inter) and h0.shape == (0, inter)


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_large_products_saturate_without_nan(nv, kind):
    """Pre-activations far past the sigmoid's range: h is g u or 0, the gradients finite."""
    m, inter, k = 16, 64, 256
    args, g, u, _, _ = operands(m, inter, k)
    args = args[:4] + (args[4] * torch.tensor([1e6, 1.0], device="cuda"),)
    g = g * 1e6
    dh = torch.ones(m, inter, dtype=torch.bfloat16, device="cuda")
    dgu, h = nv.nvfp4_gated_gemm_backward(*args, dh, activation=kind)
    assert torch.isfinite(dgu.float()).all() and torch.isfinite(h.float()).all()
    hh = h.double().cpu().numpy()
    big = np.abs(g) > 200
    ref = np.where(g > 0, g, 0.0) * u
    assert np.all(np.abs(hh - ref)[big] <= 2 * BF16 * np.abs(ref)[big] + 1e-2 * np.abs(u)[big])


def test_offsets_past_32_bits(nv):
    """More than 2^31 elements of dgu: the last rows equal those of a call on them alone (one K step, so
    every plan adds the same numbers in the same order)."""
    m, inter, k, tail = 132000, 8192, 32, 300
    ops = nvfp4_operands(512, 2 * inter, k, 6)
    b, sfb = dev(ops["qb"]), dev(ops["sfb"])
    x = torch.randn(tail, k, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    full = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    full[-tail:] = x
    gs = torch.tensor([float(ops["gsa"])], device="cuda")
    alpha = torch.tensor([float(ops["alpha"]), float(ops["alpha"])], device="cuda")
    dh = torch.ones(m, inter, dtype=torch.bfloat16, device="cuda")
    a, sfa = nv.nvfp4_quantize(full, gs)
    at, sfat = nv.nvfp4_quantize(x, gs)
    dgu, h = nv.nvfp4_gated_gemm_backward(a, sfa, b, sfb, alpha, dh)
    nv.check_status()
    want, hw = nv.nvfp4_gated_gemm_backward(at, sfat, b, sfb, alpha, dh[-tail:].contiguous())
    assert torch.equal(dgu[-tail:], want) and torch.equal(h[-tail:], hw)
    assert not dgu[: m - tail].any()
