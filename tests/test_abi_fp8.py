"""Host-side checks of the 8-bit products and the MoE gradients (no GPU needed): the entry points are exported and
refuse bad arguments before they touch a device, and the Python binding refuses what the library cannot see."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ("fp8_padded_rows", "fp8_quantize", "fp8_quantize_weight", "fp8_gemm", "fp8_grouped_gemm", "fp8_grouped_weight_grad",
         "moe_combine_backward", "moe_gather_backward")
INVALID, MISALIGNED, SHAPE = 1, 2, 3
BIG = 1 << 31


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


def test_padded_rows(nv):
    assert [nv.fp8_padded_rows(r) for r in (0, 1, 128, 129)] == [0, 128, 128, 256]
    assert nv.fp8_padded_rows(300, 4) == 384 + 512 and nv.fp8_padded_rows(0, 3) == 384
    assert nv.fp8_padded_rows(-1) == nv.fp8_padded_rows(5, -1) == 0


X, Y, W, G, O, H, S = (0x10000 * i for i in range(1, 8))   # never dereferenced: validation fails first


def test_quantize_refusals(nv):
    def call(x=X, xt=0, xr=40, k=256, ld=256, src=0, rows=40, ro=0, e=0, q=Y, sf=W, qt=0, sft=0, flags=0):
        return nv.lib.fp8_quantize(P(x), xt, xr, k, ld, P(src), rows, P(ro), e, P(q), P(sf), P(qt), P(sft), flags, None)

    both = dict(qt=G, sft=O)
    for kw, want in ((dict(xt=2), INVALID), (dict(rows=-1, xr=-1), INVALID), (dict(k=0, ld=0), INVALID), (dict(k=24, ld=24), SHAPE),
                     (dict(ld=248), MISALIGNED), (dict(ld=260), MISALIGNED), (dict(xt=1, ld=258), MISALIGNED), (dict(x=X + 8), MISALIGNED),
                     (dict(ld=-256), MISALIGNED), (dict(rows=41), INVALID), (dict(src=H, xr=-1), INVALID), (dict(q=0), INVALID),
                     (dict(sf=0), INVALID), (dict(q=0, sf=0), INVALID), (dict(qt=G), INVALID), (dict(sft=O), INVALID),
                     (dict(ro=S, e=2), INVALID), (dict(ro=S, e=0, **both), INVALID), (dict(ro=S, e=1025, **both), INVALID),
                     (dict(e=3, **both), INVALID), (dict(q=Y + 8), MISALIGNED), (dict(qt=G + 4, sft=O), MISALIGNED),
                     (dict(sf=W + 2), MISALIGNED), (dict(src=H + 2), MISALIGNED), (dict(ro=S + 4, e=2, **both), MISALIGNED),
                     (dict(x=0), INVALID), (dict(flags=2), INVALID), (dict(rows=BIG, xr=BIG), INVALID), (dict(k=BIG, ld=BIG), INVALID)):
        assert call(**kw) == want, kw
        assert nv.last_error()
    assert call(rows=0, xr=0) == 0 and call(rows=0, xr=0, x=0, q=0, sf=0) == 0


def test_quantize_weight_refusals(nv):
    def call(w=X, wt=0, e=2, n=64, k=256, ld=256, q=Y, sf=W, qt=G, sft=O, flags=0):
        return nv.lib.fp8_quantize_weight(P(w), wt, e, n, k, ld, P(q), P(sf), P(qt), P(sft), flags, None)

    for kw, want in ((dict(wt=-1), INVALID), (dict(e=-1), INVALID), (dict(n=-1), INVALID), (dict(e=1 << 20, n=1 << 20), INVALID),
                     (dict(k=40, ld=40), SHAPE), (dict(n=65), SHAPE), (dict(ld=128), MISALIGNED), (dict(w=X + 4), MISALIGNED),
                     (dict(qt=0), INVALID), (dict(sft=0), INVALID), (dict(q=0), INVALID), (dict(sf=0), INVALID), (dict(w=0), INVALID),
                     (dict(q=Y + 1), MISALIGNED), (dict(sft=O + 1), MISALIGNED), (dict(flags=4), INVALID)):
        assert call(**kw) == want, kw
    assert call(e=0) == 0 and call(n=0) == 0


def test_gemm_refusals(nv):
    def call(a=X, sa=Y, b=W, sb=G, bb=128, d=O, dt=0, acc=0, m=4, n=64, k=128, flags=0):
        return nv.lib.fp8_gemm(P(a), P(sa), P(b), P(sb), bb, P(d), dt, acc, m, n, k, flags, None)

    for kw, want in ((dict(m=-1), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(k=120), SHAPE), (dict(m=BIG), INVALID),
                     (dict(n=BIG), INVALID), (dict(k=BIG), INVALID), (dict(dt=2), INVALID), (dict(acc=1), INVALID), (dict(bb=64), INVALID),
                     (dict(flags=4), INVALID), (dict(a=0), INVALID), (dict(sa=0), INVALID), (dict(b=0), INVALID), (dict(sb=0), INVALID),
                     (dict(d=0), INVALID), (dict(a=X + 8), MISALIGNED), (dict(b=W + 1), MISALIGNED), (dict(d=O + 8), MISALIGNED),
                     (dict(sa=Y + 2), MISALIGNED), (dict(sb=G + 1), MISALIGNED)):
        assert call(**kw) == want, kw
    assert call(m=0) == 0 and call(m=0, a=0, sa=0, d=0) == 0


def test_grouped_refusals(nv):
    def rows(a=X, sa=Y, ro=H, e=2, b=W, sb=G, d=O, dt=0, t=4, n=64, k=128, flags=0):
        return nv.lib.fp8_grouped_gemm(P(a), P(sa), P(ro), e, P(b), P(sb), P(d), dt, t, n, k, flags, None)

    def grad(a=X, sa=Y, ro=H, e=2, b=W, sb=G, d=O, dt=0, acc=0, p=256, n=64, k=128, flags=0):
        return nv.lib.fp8_grouped_weight_grad(P(a), P(sa), P(b), P(sb), P(ro), e, P(d), dt, acc, p, n, k, flags, None)

    shared = [(dict(n=0), INVALID), (dict(k=0), INVALID), (dict(dt=7), INVALID), (dict(e=0), INVALID), (dict(e=1025), INVALID),
              (dict(n=1 << 30), INVALID), (dict(flags=2), INVALID), (dict(ro=0), INVALID), (dict(a=0), INVALID), (dict(sb=0), INVALID),
              (dict(d=0), INVALID), (dict(ro=H + 4), MISALIGNED), (dict(a=X + 4), MISALIGNED), (dict(d=O + 4), MISALIGNED)]
    for kw, want in shared + [(dict(t=-1), INVALID), (dict(k=24), SHAPE), (dict(t=BIG), INVALID)]:
        assert rows(**kw) == want, kw
    more = [(dict(p=0), INVALID), (dict(p=200), INVALID), (dict(p=-128), INVALID), (dict(acc=1), INVALID), (dict(p=BIG), INVALID)]
    for kw, want in [c for c in shared if "n" not in c[0] or c[0]["n"]] + more:
        assert grad(**kw) == want, kw
    assert rows(t=0) == 0


def test_moe_gradient_refusals(nv):
    def comb(do=X, ldo=64, y=Y, rows=8, pos=W, w=G, t=4, topk=2, h=64, dy=O, dw=H, flags=0):
        return nv.lib.moe_combine_backward(P(do), ldo, P(y), rows, P(pos), P(w), t, topk, h, P(dy), P(dw), flags, None)

    def gath(dxs=X, rows=8, pos=W, t=4, topk=2, h=64, dx=O, flags=0):
        return nv.lib.moe_gather_backward(P(dxs), rows, P(pos), t, topk, h, P(dx), flags, None)

    shared = [(dict(t=-1), INVALID), (dict(t=BIG), INVALID), (dict(rows=-1), INVALID), (dict(topk=0), INVALID), (dict(h=0), INVALID),
              (dict(h=60), INVALID), (dict(flags=2), INVALID), (dict(pos=0), INVALID), (dict(pos=W + 2), MISALIGNED)]
    for kw, want in shared + [(dict(ldo=56), INVALID), (dict(ldo=68), INVALID), (dict(do=0), INVALID), (dict(y=0), INVALID), (dict(w=0), INVALID),
                              (dict(dy=0), INVALID), (dict(dw=0), INVALID), (dict(dy=Y), INVALID), (dict(do=X + 8), MISALIGNED),
                              (dict(dw=H + 2), MISALIGNED)]:
        assert comb(**kw) == want, kw
    for kw, want in shared + [(dict(dxs=0), INVALID), (dict(dx=0), INVALID), (dict(dx=O + 8), MISALIGNED)]:
        assert gath(**kw) == want, kw
    assert comb(t=0, do=0) == 0 and gath(t=0, dx=0) == 0


# ------------------------------------------------------------------ the binding, against a stand-in library
@pytest.fixture()
def fake(nv, monkeypatch):
    calls = []
    real = nv._lib

    class Fake:
        fp8_padded_rows = real.fp8_padded_rows

        def __getattr__(self, name):
            def entry(*args):
                calls.append((name, args))
                return 0
            return entry

    def any_device(t, name):     # CPU tensors stand in for device tensors
        if not isinstance(t, torch.Tensor):
            raise TypeError(name)

    monkeypatch.setattr(nv, "_lib", Fake())
    monkeypatch.setattr(nv, "_check_device", any_device)
    monkeypatch.setattr(nv, "_current_device", lambda: -1)
    monkeypatch.setattr(nv, "_stream", lambda s: None)
    nv.calls = calls
    return nv


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def f32(*s):
    return torch.zeros(s)


def e4(*s):
    return torch.zeros(s, dtype=torch.uint8).view(torch.float8_e4m3fn)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def i64(*s):
    return torch.zeros(s, dtype=torch.int64)


def refused(f, **kw):
    with pytest.raises((ValueError, TypeError)):
        f(**kw)


def test_binding_quantize(fake):
    q, sf, qt, sft = fake.fp8_quantize(bf(130, 272), transpose=True)
    assert q.dtype == qt.dtype == torch.float8_e4m3fn and sf.dtype == sft.dtype == torch.float32
    assert (q.shape, sf.shape, qt.shape, sft.shape) == ((130, 272), (3, 130), (272, 256), (2, 272))
    q, sf = fake.fp8_quantize(f32(130, 272), src_rows=i32(7))
    assert q.shape == (7, 272) and sf.shape == (3, 7)
    qt, sft = fake.fp8_quantize(bf(130, 272), row_offsets=i64(5), rows=False, transpose=True)
    assert qt.shape == (272, 256 + 512) and sft.shape == (6, 272)
    fake.fp8_quantize(bf(9, 64)[:, 16:48])
    assert fake.calls[-1][1][4] == 64
    fake.fp8_quantize(bf(1, 64).expand(9, 64))
    assert fake.calls[-1][1][4] == 0
    x = bf(130, 272)
    for bad in (dict(x=x.double()), dict(x=bf(16)), dict(x=x.t()), dict(x=x, rows=False), dict(x=x, src_rows=i64(3)), dict(x=x, src_rows=i32(6)[::2]),
                dict(x=x, row_offsets=i64(3)), dict(x=x, transpose=True, row_offsets=i32(3)), dict(x=x, transpose=True, row_offsets=i64(1)),
                dict(x=x, transpose=True, row_offsets=i64(6)[::2]), dict(x=x, q=e4(130, 256)), dict(x=x, q=bf(130, 272)), dict(x=x, sf=f32(130, 3)),
                dict(x=x, qt=e4(272, 256)), dict(x=x, rows=False, transpose=True, q=e4(130, 272)), dict(x=x, transpose=True, sft=f32(1, 272))):
        refused(fake.fp8_quantize, **bad)


def test_binding_quantize_weight(fake):
    q, sf, qt, sft = fake.fp8_quantize_weight(f32(3, 144, 272), transpose=True)
    assert (q.shape, sf.shape, qt.shape, sft.shape) == ((3, 144, 272), (3, 2, 3), (3, 272, 144), (3, 3, 2))
    assert fake.fp8_quantize_weight(bf(144, 288)[:, :272])[1].shape == (2, 3) and fake.calls[-1][1][5] == 288
    for bad in (dict(w=f32(3)), dict(w=f32(3, 144, 272).transpose(1, 2)), dict(w=f32(4, 4).half()), dict(w=f32(144, 272), qt=e4(272, 144)),
                dict(w=f32(144, 272), q=e4(144, 256)), dict(w=f32(144, 272), sf=f32(3, 2))):
        refused(fake.fp8_quantize_weight, **bad)


def test_binding_products(fake):
    m, n, k = 5, 200, 272
    args = dict(a=e4(m, k), sfa=f32(3, m), b=e4(n, k), sfb=f32(2, 3))
    assert fake.fp8_gemm(**args).dtype == torch.bfloat16 and fake.fp8_gemm(**args).shape == (m, n)
    assert fake.fp8_gemm(**{**args, "sfb": f32(3, n)}, block_b=1, out_dtype=torch.float32).dtype == torch.float32
    d = f32(m, n)
    assert fake.fp8_gemm(**args, d=d, accumulate=True) is d and fake.calls[-1][1][6:8] == (1, 1)
    for bad in (dict(a=e4(m, 256)), dict(a=bf(m, k)), dict(a=e4(k, m).t()), dict(sfa=f32(m, 3)), dict(sfb=f32(3, 2)), dict(sfb=f32(3, n)),
                dict(block_b=1), dict(block_b=64), dict(out_dtype=torch.float16), dict(accumulate=True), dict(d=f32(n, m)), dict(d=f32(m, 2 * n)[:, ::2]),
                dict(b=e4(k, n).t()), dict(sfa=bf(3, m))):
        refused(fake.fp8_gemm, **{**args, **bad})
    g = dict(a=e4(m, k), sfa=f32(3, m), row_offsets=i64(5), b=e4(4, n, k), sfb=f32(4, 2, 3))
    assert fake.fp8_grouped_gemm(**g).shape == (m, n)
    for bad in (dict(row_offsets=i64(4)), dict(row_offsets=i32(5)), dict(row_offsets=i64(10)[::2]), dict(b=e4(n, k)), dict(sfb=f32(4, 3, 2)),
                dict(sfa=f32(3, 4)), dict(d=bf(m + 1, n)), dict(a=e4(m, 256))):
        refused(fake.fp8_grouped_gemm, **{**g, **bad})
    w = dict(a=e4(n, 640), sfa=f32(5, n), b=e4(k, 640), sfb=f32(5, k), row_offsets=i64(5))
    assert fake.fp8_grouped_weight_grad(**w).shape == (4, n, k)
    for bad in (dict(b=e4(k, 512)), dict(sfa=f32(n, 5)), dict(sfb=f32(4, k)), dict(row_offsets=i32(5)), dict(accumulate=True), dict(d=f32(4, k, n)),
                dict(d=bf(4, n, k), accumulate=False, out_dtype=None, a=bf(n, 640))):
        refused(fake.fp8_grouped_weight_grad, **{**w, **bad})


def test_binding_moe_gradients(fake):
    args = dict(dout=bf(4, 64), y=bf(9, 64), pos=i32(4, 2), weights=f32(4, 2))
    dy, dw = fake.moe_combine_backward(**args)
    assert dy.shape == (9, 64) and dy.dtype == torch.bfloat16 and dw.shape == (4, 2) and dw.dtype == torch.float32
    fake.moe_combine_backward(**{**args, "dout": bf(1, 64).expand(4, 64), "pos": i32(2, 4).t(), "weights": f32(2, 4).t()})
    assert fake.calls[-1][1][1] == 0
    for bad in (dict(dout=bf(4, 56)), dict(dout=f32(4, 64)), dict(y=bf(64, 9).t()), dict(pos=i64(4, 2)), dict(weights=f32(4, 3)), dict(weights=bf(4, 2)),
                dict(dy=bf(8, 64)), dict(dweights=f32(8))):
        refused(fake.moe_combine_backward, **{**args, **bad})
    assert fake.moe_gather_backward(bf(9, 64), i32(4, 2)).shape == (4, 64)
    for bad in (dict(dxs=f32(9, 64)), dict(dxs=bf(64, 9).t()), dict(pos=i64(4, 2)), dict(pos=i32(8)), dict(dx=bf(5, 64))):
        refused(fake.moe_gather_backward, **{**dict(dxs=bf(9, 64), pos=i32(4, 2)), **bad})
