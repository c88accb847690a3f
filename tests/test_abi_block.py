"""Host-side checks of the decoder-block entry points (no GPU needed): they are exported, answer their size
queries and refuse bad arguments before they touch a device, and the Python binding refuses what the
library cannot see."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ("block_norm", "block_norm_quantize", "block_norm_backward", "block_norm_backward_workspace_size",
         "nvfp4_gated_gemm", "nvfp4_gated_gemm_backward", "sample_tokens")
INVALID, MISALIGNED, SHAPE = 1, 2, 3


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_bf16_gb300 as m
    return m


def P(v):
    return ctypes.c_void_p(v) if v else None


def test_declared_and_exported(nv):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "nvfp4.h")).read(), flags=re.S)
    raw = ctypes.CDLL(nv.LIB_PATH)
    for name in NAMES:
        assert re.search(r"\b%s\s*\(" % name, text), name
        assert hasattr(raw, name), name


# never dereferenced: validation fails first
X, Y, W, G, O, H, S = (0x10000 * i for i in range(1, 8))


def test_block_norm_refusals(nv):
    def call(x=X, xt=0, ldx=64, y=Y, ldy=64, wpost=W, gate=G, ldg=0, wpre=W, xo=O, ldxo=64, h=H, ldh=64, m=4, n=64, flags=0):
        return nv.lib.block_norm(P(x), xt, ldx, P(y), ldy, P(wpost), P(gate), ldg, P(wpre), 1.0, 1e-6, 0.0, P(xo), ldxo, P(h),
                                 ldh, m, n, flags, None)

    for kw, want in ((dict(m=-1), INVALID), (dict(n=0), INVALID), (dict(n=32769, ldx=40000, ldy=40000, ldxo=40000, ldh=40000), SHAPE),
                     (dict(m=1 << 31), INVALID), (dict(xt=2), INVALID), (dict(flags=1 << 2), INVALID), (dict(x=0), INVALID),
                     (dict(xo=0), INVALID), (dict(ldx=63), INVALID), (dict(ldx=-64), INVALID), (dict(ldy=10), INVALID),
                     (dict(ldg=8), INVALID), (dict(ldxo=0), INVALID), (dict(ldh=32), INVALID), (dict(h=0), INVALID),
                     (dict(wpre=0), INVALID), (dict(y=0), INVALID), (dict(y=0, wpost=0, gate=0, xo=0, wpre=0, h=0), INVALID),
                     (dict(y=0, wpost=0), INVALID), (dict(x=X + 1), MISALIGNED), (dict(xt=1, x=X + 2), MISALIGNED),
                     (dict(gate=G + 1), MISALIGNED), (dict(h=H + 1), MISALIGNED)):
        assert call(**kw) == want, kw
        assert nv.last_error()
    assert call(m=0) == 0 and call(m=0, x=0, y=0, wpost=0, gate=0, wpre=0, xo=0, h=0) == 0


def test_block_norm_quantize_refusals(nv):
    def call(x=X, ldx=64, wpre=W, gs=S, q=H, sf=G, n=64, m=4, xo=O, y=Y, flags=0):
        return nv.lib.block_norm_quantize(P(x), 0, ldx, P(y), 64, None, None, 0, P(wpre), 1.0, 1e-6, 0.0, P(xo), 64, P(gs), P(q),
                                          P(sf), m, n, flags, None)

    for kw, want in ((dict(n=40), SHAPE), (dict(wpre=0), INVALID), (dict(gs=0), INVALID), (dict(q=0), INVALID), (dict(sf=0), INVALID),
                     (dict(x=X + 8), MISALIGNED), (dict(ldx=68), MISALIGNED), (dict(wpre=W + 2), MISALIGNED),
                     (dict(sf=G + 8), MISALIGNED), (dict(q=H + 4), MISALIGNED), (dict(gs=S + 2), MISALIGNED),
                     (dict(flags=1 << 9), INVALID)):
        assert call(**kw) == want, kw
    assert call(m=0) == 0


def test_block_norm_backward_refusals(nv):
    need = nv.block_norm_backward_workspace_size(4, 64)

    def call(dh=X, dr=X, r=X, xt=0, ld=64, y=Y, wpost=W, gate=G, ldg=0, wpre=W, dx=O, dy=O, dwpre=H, dwpost=H, dgate=H, lddg=0,
             m=4, n=64, ws=S, wsb=None, flags=0, lddx=64):
        return nv.lib.block_norm_backward(P(dh), ld, P(dr), ld, P(r), xt, ld, P(y), ld, P(wpost), P(gate), ldg, P(wpre), 1.0,
                                          1e-6, 0.0, P(dx), lddx, P(dy), 64, P(dwpre), P(dwpost), P(dgate), lddg, m, n, P(ws),
                                          need if wsb is None else wsb, flags, None)

    for kw, want in ((dict(m=-1), INVALID), (dict(n=0), INVALID), (dict(xt=7), INVALID), (dict(flags=4), INVALID),
                     (dict(ld=32), INVALID), (dict(lddx=0), INVALID), (dict(dh=0), INVALID), (dict(wpre=0), INVALID),
                     (dict(dwpre=0), INVALID), (dict(dwpost=0), INVALID), (dict(dgate=0), INVALID), (dict(gate=0), INVALID),
                     (dict(y=0), INVALID), (dict(dy=0), INVALID), (dict(r=0), INVALID), (dict(dx=0), INVALID),
                     (dict(ldg=64, lddg=8), INVALID), (dict(ws=0), INVALID), (dict(wsb=need - 1), INVALID),
                     (dict(ws=S + 8), MISALIGNED), (dict(dx=O + 1), MISALIGNED), (dict(dwpre=H + 2), MISALIGNED),
                     (dict(n=32776, ld=40000, lddx=40000), SHAPE)):
        assert call(**kw) == want, kw
    assert "workspace" in (call(wsb=0) and nv.last_error())


def test_backward_workspace_size(nv):
    """Three rows of fp32 sums per team; no more teams than rows."""
    f = nv.block_norm_backward_workspace_size
    assert f(0, 64) == 0 and f(1, 64) == 3 * 64 * 4 and f(7, 4096) == 7 * 3 * 4096 * 4
    assert f(-1, 64) == 0 and f(4, 0) == 0 and f(4, 40000) == 0
    for n in (16, 512, 520, 1024, 2048, 4096, 8192, 32768):
        assert f(1 << 20, n) % (12 * n) == 0 and f(1 << 20, n) == f(1 << 21, n) >= f(1000, n)


def test_gated_refusals(nv):
    A, SA, B, SB, AL, D, DH = X, Y, W, G, S, O, H

    def fwd(a=A, sfa=SA, b=B, sfb=SB, alpha=AL, act=0, h=D, m=32, inter=64, k=128, flags=0):
        return nv.lib.nvfp4_gated_gemm(P(a), P(sfa), P(b), P(sfb), P(alpha), act, P(h), m, inter, k, None, 0, flags, None)

    def bwd(dh=DH, dgu=D, h=D, m=32, inter=64, k=128, act=1):
        return nv.lib.nvfp4_gated_gemm_backward(P(A), P(SA), P(B), P(SB), P(AL), act, P(dh), P(dgu), P(h), m, inter, k, None, 0, 0, None)

    for kw, want in ((dict(inter=0), INVALID), (dict(inter=24), SHAPE), (dict(k=100), SHAPE), (dict(act=2), INVALID),
                     (dict(act=-1), INVALID), (dict(m=-1), INVALID), (dict(a=0), INVALID), (dict(b=0), INVALID),
                     (dict(alpha=0), INVALID), (dict(h=0), INVALID), (dict(h=D + 16), MISALIGNED), (dict(a=A + 16), MISALIGNED),
                     (dict(sfb=SB + 8), MISALIGNED), (dict(flags=1 << 20), INVALID), (dict(inter=1 << 30), INVALID)):
        assert fwd(**kw) == want, kw
    for kw, want in ((dict(dh=0), INVALID), (dict(dgu=0), INVALID), (dict(dh=DH + 16), MISALIGNED), (dict(h=D + 8), MISALIGNED),
                     (dict(inter=8), SHAPE), (dict(act=9), INVALID)):
        assert bwd(**kw) == want, kw
    # split plans refuse a missing workspace by name
    assert nv.lib.nvfp4_gated_gemm(P(A), P(SA), P(B), P(SB), P(AL), 0, P(D), 0, 64, 128, None, 0, 0, None) == 0


def test_sample_refusals(nv):
    def call(z=X, zt=0, ld=100, u=Y, t=0, k=0, p=0, mp=0, tok=O, lp=0, rows=4, v=100, flags=0):
        return nv.lib.sample_tokens(P(z), zt, ld, P(u), P(t), P(k), P(p), P(mp), P(tok), P(lp), rows, v, flags, None)

    for kw, want in ((dict(rows=-1), INVALID), (dict(v=0), INVALID), (dict(v=(1 << 21) + 1, ld=1 << 22), SHAPE), (dict(zt=3), INVALID),
                     (dict(ld=99), INVALID), (dict(ld=-100), INVALID), (dict(z=0), INVALID), (dict(u=0), INVALID), (dict(tok=0), INVALID),
                     (dict(z=X + 1), MISALIGNED), (dict(zt=1, z=X + 2), MISALIGNED), (dict(k=W + 2), MISALIGNED),
                     (dict(tok=O + 2), MISALIGNED), (dict(flags=2), INVALID), (dict(rows=1 << 28), INVALID)):
        assert call(**kw) == want, kw
    assert call(rows=0, z=0, u=0, tok=0) == 0


# ------------------------------------------------------------------ the binding, against a stand-in library
@pytest.fixture()
def fake(nv, monkeypatch):
    calls = []
    real = nv._lib

    class Fake:
        nvfp4_sf_bytes = real.nvfp4_sf_bytes
        block_norm_backward_workspace_size = real.block_norm_backward_workspace_size

        def __getattr__(self, name):
            def entry(*args):
                calls.append((name, args))
                return 0
            return entry

    monkeypatch.setattr(nv, "_lib", Fake())
    def any_device(t, name):     # CPU tensors stand in for device tensors
        if not isinstance(t, torch.Tensor):
            raise TypeError(name)

    monkeypatch.setattr(nv, "_check_device", any_device)
    monkeypatch.setattr(nv, "_stream", lambda s: None)
    nv.calls = calls
    return nv


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def f32(*s):
    return torch.zeros(s)


def test_binding_block_norm(fake):
    x, y, w = bf(3, 40), bf(3, 40), bf(40)
    x_out, h = fake.block_norm(x, w, y=y, w_post=w, gate=w)
    assert x_out.shape == h.shape == (3, 40) and x_out is not x
    same, h = fake.block_norm(x, w)
    assert same is x and h.dtype == torch.bfloat16
    out, none = fake.block_norm(f32(3, 40), None, y=y)
    assert none is None and out.dtype == torch.float32
    fake.block_norm(bf(3, 64)[:, 8:48], w, y=y)                      # rows of a wider buffer
    assert fake.calls[-1][1][2] == 64
    fake.block_norm(x[:1].expand(3, 40), w)                          # one row for all
    assert fake.calls[-1][1][2] == 0
    fake.block_norm(x, w, y=y, gate=bf(1, 40).expand(3, 40))         # a gate per token, laid out
    assert fake.calls[-1][1][7] == 40
    for bad in (dict(y=bf(3, 41)), dict(y=f32(3, 40)), dict(y=y, w_post=bf(41)), dict(y=y, w_post=f32(40)), dict(w_post=w),
                dict(gate=w), dict(y=y, gate=bf(2, 40)), dict(y=y, x_out=f32(3, 40)), dict(y=y, h=bf(3, 39)), dict(x_out=x),
                dict(y=bf(40, 3).t()), dict(y=[1.0])):
        with pytest.raises((ValueError, TypeError)):
            fake.block_norm(x, w, **bad)
    with pytest.raises(TypeError):
        fake.block_norm(x.double(), w)
    with pytest.raises(ValueError):
        fake.block_norm(bf(40), w)
    with pytest.raises(ValueError):
        fake.block_norm(x, None, y=y, h=bf(3, 40))


def test_binding_block_norm_quantize_and_backward(fake):
    x, y, w = bf(3, 48), bf(3, 48), bf(48)
    x_out, q, sf = fake.block_norm_quantize(x, w, f32(1), y=y)
    assert q.shape == (3, 24) and sf.numel() == fake.sf_bytes(3, 48)
    for bad in (dict(q=torch.zeros(3, 23, dtype=torch.uint8)), dict(sf=torch.zeros(4, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            fake.block_norm_quantize(x, w, f32(1), **bad)
    with pytest.raises(TypeError):
        fake.block_norm_quantize(x, w, bf(1))
    with pytest.raises(ValueError):
        fake.block_norm_quantize(x, None, f32(1))
    dx, dy, a, b, g = fake.block_norm_backward(x, None, x, w, y=y, w_post=w, gate=w)
    assert dx.shape == dy.shape == (3, 48) and a.shape == b.shape == g.shape == (48,) and g.dtype == torch.float32
    g = fake.block_norm_backward(x, x, x, w, y=y, gate=bf(3, 48))[4]
    assert g.shape == (3, 48) and g.dtype == torch.bfloat16
    dx, dy, a, b, g = fake.block_norm_backward(x, x, x, w)
    assert dy is None and a.shape == (48,) and b is None and g is None
    for bad in (dict(dh=None), dict(dh=f32(3, 48)), dict(dx_out=f32(3, 48)), dict(dx_out=bf(2, 48))):
        with pytest.raises((ValueError, TypeError)):
            fake.block_norm_backward(**{**dict(dh=x, dx_out=x, x_out=x, w_pre=w), **bad})


def test_binding_gated(fake):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    m, inter, k = 5, 32, 64
    a, b = u8(m, k // 2), u8(2 * inter, k // 2)
    args = (a, u8(fake.sf_bytes(m, k)), b, u8(fake.sf_bytes(2 * inter, k)), f32(2))
    assert fake.nvfp4_gated_gemm(*args).shape == (m, inter)
    dgu, h = fake.nvfp4_gated_gemm_backward(*args, bf(m, inter), activation="gelu_tanh")
    assert dgu.shape == (m, 2 * inter) and h.shape == (m, inter)
    for i, bad in ((0, u8(m, 31)), (1, u8(3)), (2, u8(2 * inter, 16)), (3, u8(3)), (4, f32(1)), (4, bf(2))):
        with pytest.raises((ValueError, TypeError)):
            fake.nvfp4_gated_gemm(*args[:i], bad, *args[i + 1:])
    with pytest.raises(ValueError):
        fake.nvfp4_gated_gemm(*args, activation="relu")
    with pytest.raises(ValueError):
        fake.nvfp4_gated_gemm(*args, h=bf(m, inter - 1))
    for bad in (bf(m, inter + 1), f32(m, inter), bf(inter)):
        with pytest.raises((ValueError, TypeError)):
            fake.nvfp4_gated_gemm_backward(*args, bad)


def test_binding_interleave(nv):
    g = torch.arange(32 * 3).view(32, 3)
    w = nv.interleave_gate_up(g, -g)
    assert torch.equal(w[:16], g[:16]) and torch.equal(w[16:32], -g[:16]) and torch.equal(w[32:48], g[16:])
    for a, b in ((g[:20], g[:20]), (g, g[:16])):
        with pytest.raises(ValueError):
            nv.interleave_gate_up(a, b)


def test_binding_sample(fake):
    z, u = bf(3, 50), f32(3)
    tok, lp = fake.sample_tokens(z, u, top_k=torch.zeros(3, dtype=torch.int32))
    assert tok.shape == lp.shape == (3,) and tok.dtype == torch.int32
    fake.sample_tokens(f32(3, 60)[:, 3:53], u)
    assert fake.calls[-1][1][2] == 60
    for bad in (dict(uniform=None), dict(uniform=f32(2)), dict(uniform=bf(3)), dict(top_k=f32(3)), dict(top_p=f32(3, 1)),
                dict(min_p=f32(6)[::2]), dict(temperature=f32(4)), dict(tokens=f32(3)), dict(logprobs=f32(4))):
        with pytest.raises((ValueError, TypeError)):
            fake.sample_tokens(**{**dict(logits=z, uniform=u), **bad})
    for bad in (z.double(), bf(50), z.t()):
        with pytest.raises((ValueError, TypeError)):
            fake.sample_tokens(bad, u)
