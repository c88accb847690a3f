"""The feed-forward half of a decoder on the library's NVFP4 products, from the residual stream to the next
token, and its backward pass.

    python examples/decoder_step.py [--tokens 8] [--layers 4] [--hidden 4096] [--inter 7168] [--vocab 32768]

A layer keeps the stream x [tokens, hidden] and runs

    x, a = stream + norm after the last block, norm before this one, NVFP4   block_norm_quantize
    h    = silu(a Wg^T) * (a Wu^T)                                           nvfp4_gated_gemm
    y    = h Wd^T                                                            nvfp4_quantize, nvfp4_gemm

then the head's product gives logits and sample_tokens draws from them.  Weights are random and laid out once;
the activations' global scales are calibrated on the first step, as a serving engine would.  Attention is
left out: the library has none.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_block_scaled_bf16_gb300 as nv  # noqa: E402


def _global_scale(t: torch.Tensor) -> torch.Tensor:
    """448 * 6 / amax, the global scale under which t's largest block just fits."""
    return (2688.0 / t.float().abs().amax().clamp(min=1e-12)).reshape(1)


class Weight:
    """A [n, k] bf16 weight as NVFP4, and its transpose for the backward pass where asked for."""

    def __init__(self, w: torch.Tensor, transpose: bool = False):
        self.gs = _global_scale(w)
        self.q, self.sf = nv.nvfp4_quantize(w, self.gs)
        self.t = Weight(w.t().contiguous()) if transpose else None

    def product(self, x: torch.Tensor, gs: torch.Tensor | None = None, flags: int = 0) -> torch.Tensor:
        """x W^T for a bf16 x: quantise, multiply."""
        gs = _global_scale(x) if gs is None else gs
        a, sfa = nv.nvfp4_quantize(x, gs, flags=flags)
        return nv.nvfp4_gemm(a, sfa, self.q, self.sf, 1.0 / (gs * self.gs), flags=flags)


class Layer:
    def __init__(self, hidden: int, inter: int, gen: torch.Generator, train: bool):
        def normal(*shape, std=0.02):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)

        self.gate_up = Weight(nv.interleave_gate_up(normal(inter, hidden), normal(inter, hidden)), train)
        self.down = Weight(normal(hidden, inter), train)
        self.w_pre = 1.0 + normal(hidden, std=0.05)
        self.w_post = 1.0 + normal(hidden, std=0.05)
        self.gs_a = self.gs_h = None       # calibrated on the first step


class Decoder:
    def __init__(self, layers: int = 4, hidden: int = 4096, inter: int = 7168, vocab: int = 32768, seed: int = 0,
                 residual_scale: float = 1.0, train: bool = False):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [Layer(hidden, inter, gen, train) for _ in range(layers)]
        self.w_final = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
        self.head = Weight((torch.randn(vocab, hidden, generator=gen, device="cuda") * 0.02).to(torch.bfloat16))
        self.residual_scale = residual_scale
        self.gs_final = None

    def _calibrate(self, x: torch.Tensor) -> None:
        """The activations' global scales and the products' alphas, from one pass through the layers."""
        y = w_post = None
        for la in self.layers:
            x, a = nv.block_norm(x, la.w_pre, y=y, w_post=w_post, residual_scale=self.residual_scale)
            la.gs_a = _global_scale(a)
            q, sf = nv.nvfp4_quantize(a, la.gs_a)
            la.alpha = (1.0 / (la.gs_a * la.gate_up.gs)).repeat(2)
            h = nv.nvfp4_gated_gemm(q, sf, la.gate_up.q, la.gate_up.sf, la.alpha)
            la.gs_h = _global_scale(h)
            la.alpha_down = 1.0 / (la.gs_h * la.down.gs)
            y, w_post = la.down.product(h, la.gs_h), la.w_post
        self.gs_final = _global_scale(nv.block_norm(x, self.w_final, y=y, w_post=w_post, residual_scale=self.residual_scale)[1])
        self.alpha_head = 1.0 / (self.gs_final * self.head.gs)

    def logits(self, x: torch.Tensor, flags: int = nv.FLAG_PDL) -> torch.Tensor:
        """bf16 [tokens, vocab] from the stream x; every kernel launched with PDL behind the one before."""
        if self.gs_final is None:
            self._calibrate(x)
        y = w_post = None
        for la in self.layers:
            x, a, sfa = nv.block_norm_quantize(x, la.w_pre, la.gs_a, y=y, w_post=w_post,
                                               residual_scale=self.residual_scale, flags=flags)
            h = nv.nvfp4_gated_gemm(a, sfa, la.gate_up.q, la.gate_up.sf, la.alpha, flags=flags)
            q, sf = nv.nvfp4_quantize(h, la.gs_h, flags=flags)
            y = nv.nvfp4_gemm(q, sf, la.down.q, la.down.sf, la.alpha_down, flags=flags)
            w_post = la.w_post
        x, a, sfa = nv.block_norm_quantize(x, self.w_final, self.gs_final, y=y, w_post=w_post,
                                           residual_scale=self.residual_scale, flags=flags)
        return nv.nvfp4_gemm(a, sfa, self.head.q, self.head.sf, self.alpha_head, flags=flags)

    def step(self, x, uniform, temperature=None, top_k=None, top_p=None, min_p=None):
        """The next token of every row of x: (tokens int32, log-probabilities fp32)."""
        return nv.sample_tokens(self.logits(x), uniform, temperature, top_k, top_p, min_p, flags=nv.FLAG_PDL)


def block_gradients(la: Layer, x: torch.Tensor, d_out: torch.Tensor, residual_scale: float = 1.0):
    """Forward and backward pass of one block, out = x + scale * norm(ffn(norm(x))): returns (out, dx, and the
    gradients of the two norms' weights).  The four products of the backward pass run in NVFP4 too, from the
    transposed weights."""
    _, a = nv.block_norm(x, la.w_pre)
    gs = _global_scale(a)
    q, sf = nv.nvfp4_quantize(a, gs)
    alpha = (1.0 / (gs * la.gate_up.gs)).repeat(2)
    h = nv.nvfp4_gated_gemm(q, sf, la.gate_up.q, la.gate_up.sf, alpha)
    y = la.down.product(h)
    out, _ = nv.block_norm(x, None, y=y, w_post=la.w_post, residual_scale=residual_scale)
    # backward: the norm after the block and the sum, the down product, the gated product (its two products
    # again from the packed operands), the product with both projections, the norm before the block
    dx, dy, _, dw_post, _ = nv.block_norm_backward(None, d_out, out, None, y=y, w_post=la.w_post,
                                                   residual_scale=residual_scale)
    dh = la.down.t.product(dy)
    dgu, _ = nv.nvfp4_gated_gemm_backward(q, sf, la.gate_up.q, la.gate_up.sf, alpha, dh)
    da = la.gate_up.t.product(dgu)
    dx, _, dw_pre, _, _ = nv.block_norm_backward(da, dx, x, la.w_pre)
    return out, dx, dw_pre, dw_post


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 8), ("layers", 4), ("hidden", 4096), ("inter", 7168), ("vocab", 32768), ("steps", 50)):
        ap.add_argument(f"--{name}", type=int, default=value)
    args = ap.parse_args()
    model = Decoder(args.layers, args.hidden, args.inter, args.vocab)
    n = args.tokens
    x = torch.randn(n, args.hidden, device="cuda").to(torch.bfloat16)
    u = torch.rand(n, device="cuda")
    opts = dict(temperature=torch.full((n,), 0.8, device="cuda"), top_k=torch.full((n,), 50, dtype=torch.int32, device="cuda"),
                top_p=torch.full((n,), 0.95, device="cuda"), min_p=torch.full((n,), 0.02, device="cuda"))
    model.step(x, u, **opts)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens, logprobs = model.step(x, u, **opts)
    for _ in range(5):
        graph.replay()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(args.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    nv.check_status()
    print(f"{n} tokens, {args.layers} layers of {args.hidden} x {args.inter}, vocabulary {args.vocab}: "
          f"{begin.elapsed_time(end) / args.steps * 1e3:.1f} us a step")
    print("tokens  ", tokens.tolist())
    print("logprobs", [round(v, 3) for v in logprobs.tolist()])


if __name__ == "__main__":
    main()
