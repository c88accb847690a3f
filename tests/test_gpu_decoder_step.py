"""The decoder example: its steps against the same layer put together from the library's other calls, its
gradients against a plain fp32 layer on the dequantised weights."""
import os
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    import __graft_entry__
    __graft_entry__.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decoder_step
    return decoder_step


def test_step_equals_its_pieces(ex):
    """block_norm_quantize is block_norm then nvfp4_quantize bit for bit, and PDL changes nothing, so the
    logits of the fused steps equal those of the separate ones; the token is drawn from them."""
    nv = ex.nv
    model = ex.Decoder(layers=2, hidden=512, inter=768, vocab=2048, seed=3, residual_scale=0.5)
    x0 = torch.randn(19, 512, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    logits = model.logits(x0)
    x, y, w_post = x0, None, None
    for la in model.layers:
        x, a = nv.block_norm(x, la.w_pre, y=y, w_post=w_post, residual_scale=0.5)
        q, sf = nv.nvfp4_quantize(a, la.gs_a)
        h = nv.nvfp4_gated_gemm(q, sf, la.gate_up.q, la.gate_up.sf, la.alpha)
        y, w_post = la.down.product(h, la.gs_h), la.w_post
    _, a = nv.block_norm(x, model.w_final, y=y, w_post=w_post, residual_scale=0.5)
    assert torch.equal(logits, model.head.product(a, model.gs_final))
    u = torch.rand(19, generator=torch.Generator().manual_seed(2)).cuda()
    p = torch.full((19,), 0.9, device="cuda")
    tokens, logprobs = model.step(x0, u, top_p=p)
    want, lp = nv.sample_tokens(logits, u, top_p=p)
    assert torch.equal(tokens, want) and torch.equal(logprobs, lp)
    nv.check_status()


def test_step_in_a_graph(ex):
    """Captured once, replayed with new inputs in place."""
    nv = ex.nv
    model = ex.Decoder(layers=2, hidden=1024, inter=512, vocab=4096, seed=4)
    x = torch.randn(4, 1024, device="cuda").to(torch.bfloat16)
    u = torch.tensor([0.1, 0.4, 0.6, 0.9], device="cuda")
    k = torch.full((4,), 40, dtype=torch.int32, device="cuda")
    model.step(x, u, top_k=k)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tokens, _ = model.step(x, u, top_k=k)
    for seed in (5, 6):
        x.copy_(torch.randn(4, 1024, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        got = tokens.clone()
        assert torch.equal(got, model.step(x, u, top_k=k)[0])
    nv.check_status()


def test_block_gradients(ex):
    """Against autograd through the layer in fp32 on unquantised random weights: 4-bit products carry about
    10 % noise an element (e2m1 steps are up to 1/4 of a value, averaged over a block), so the gradients are
    compared as directions: the noise of four products in a row keeps the cosine above 0.9, while a
    missing term, factor or transposition does not."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    hidden, inter, m = 512, 768, 200
    made = []
    weight = ex.Weight

    class Kept(weight):
        def __init__(self, w, transpose=False):
            made.append(w.float())
            super().__init__(w, transpose)

    ex.Weight = Kept
    try:
        la = ex.Layer(hidden, inter, gen, train=True)
    finally:
        ex.Weight = weight
    gu, down = made[0], made[2]
    x = torch.randn(m, hidden, generator=gen, device="cuda").to(torch.bfloat16)
    d_out = (torch.randn(m, hidden, generator=gen, device="cuda") * 0.1).to(torch.bfloat16)
    out, dx, dw_pre, dw_post = ex.block_gradients(la, x, d_out, 0.7)
    xs = x.float().requires_grad_()
    wp, wq = la.w_pre.float().requires_grad_(), la.w_post.float().requires_grad_()

    def rms(v, w):
        return v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * w

    c = (rms(xs, wp) @ gu.t()).view(m, -1, 2, 16)
    h = (torch.nn.functional.silu(c[:, :, 0]) * c[:, :, 1]).reshape(m, inter)
    ref = xs + 0.7 * rms(h @ down.t(), wq)
    ref.backward(d_out.float())
    branch = (dx.float() - d_out.float(), xs.grad - d_out.float())       # without the residual path
    for a, b in ((out.float() - x.float(), (ref - xs).detach()), branch, (dw_pre, wp.grad), (dw_post, wq.grad)):
        cos = torch.nn.functional.cosine_similarity(a.reshape(1, -1), b.reshape(1, -1)).item()
        ratio = (a.norm() / b.norm()).item()
        assert cos > 0.9 and 0.8 < ratio < 1.25, (cos, ratio)
