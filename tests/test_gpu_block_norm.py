"""The norms around a decoder block on the GPU against the fp64 forms of oracle/block.py.

Bounds, fixed by the arithmetic.  A bf16 result is rounded once: half a bf16 ulp, at most 2^-8 of the
value.  The fp32 arithmetic before it: a row sum adds at most 32 values per thread in a chain, then
trees of at most 10 levels, so every mean carries a relative error below 48 * 2^-24 < 2^-18 of the sum
of magnitudes, and the few products around it a handful of 2^-24 each; FP32 = 2^-17 of the sum of the
magnitudes that enter a result covers both.  A column sum is a chain of at most m / teams rows, then
of teams / 128 + 32 + 32 partial sums: below 128 additions in these tests, 2^-17 again."""
import numpy as np
import pytest
import torch

from oracle import block
from oracle import quant as oquant

pytestmark = pytest.mark.gpu

BF16, FP32 = 2.0 ** -8, 2.0 ** -17
EPS = 1e-6


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_bf16_gb300 as m
    return m


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def inputs(m, n, stream=torch.bfloat16, post=True, gate="channel", seed=0, pad=0):
    g = torch.Generator().manual_seed(seed + 31 * m + n)

    def rows(dtype, std):
        full = (torch.randn(m, n + pad, generator=g) * std).to(dtype).cuda()
        return full[:, :n]

    d = dict(x=rows(stream, 1.0), y=None, w_post=None, gate=None)
    if n >= 4:
        d["x"][:, n // 4] *= 20
    vec = lambda std, mean: (mean + torch.randn(n, generator=g) * std).to(torch.bfloat16).cuda()  # noqa: E731
    d["w_pre"] = vec(0.2, 1.0)
    if post is not None:
        d["y"] = rows(torch.bfloat16, 0.7)
        d["w_post"] = vec(0.2, 1.0) if post else None
        d["gate"] = {"none": None, "channel": vec(0.5, 0.0), "token": rows(torch.bfloat16, 0.5)}[gate]
    d["dh"] = rows(torch.bfloat16, 0.1)
    d["dr"] = rows(stream, 0.1)
    return d


def check(got, ref, rounding, terms, what):
    got = f64(got)
    tol = rounding * np.abs(ref) + FP32 * terms + 1e-30
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside, worst {np.max(np.abs(got - ref) / tol):.3g} of the bound"


def forward_terms(d, scale, offset):
    """Magnitudes that enter r and h."""
    x = np.abs(f64(d["x"]))
    r, _ = block.block_norm(f64(d["x"]), None, f64(d["y"]), f64(d["w_post"]), f64(d["gate"]), scale, EPS, offset)
    tr = x if d["y"] is None else x + np.abs(r - f64(d["x"]))
    rstd = 1.0 / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + EPS)
    th = None if d["w_pre"] is None else (tr + np.abs(r)) * rstd * np.abs(offset + f64(d["w_pre"]))
    return tr, th


SHAPES = [(1, 1), (1, 7), (3, 8), (1, 16), (5, 255), (9, 256), (4, 257), (2, 512), (3, 520), (700, 96), (1, 2047),
          (6, 2048), (77, 2047), (1, 7168), (700, 4096), (2, 8200), (2, 12296), (3, 20000), (2, 32768),
          # from 4 rows an SM on, aligned rows are copied ahead
          (608, 520), (700, 1032), (613, 2056), (1300, 4104), (620, 7168), (609, 8192), (640, 10248), (650, 7177)]


@pytest.mark.parametrize("m,n", SHAPES)
def test_forward(nv, m, n):
    d = inputs(m, n)
    x_out, h = nv.block_norm(d["x"], d["w_pre"], y=d["y"], w_post=d["w_post"], gate=d["gate"], residual_scale=0.7, eps=EPS)
    r_ref, h_ref = block.block_norm(f64(d["x"]), f64(d["w_pre"]), f64(d["y"]), f64(d["w_post"]), f64(d["gate"]), 0.7, EPS)
    tr, th = forward_terms(d, 0.7, 0.0)
    check(x_out, r_ref, BF16, tr, "x_out")
    check(h, h_ref, BF16, th, "h")


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("post,gate", [(True, "none"), (True, "channel"), (True, "token"), (False, "none"), (False, "channel"),
                                       (False, "token"), (None, "none")])
@pytest.mark.parametrize("m,n,pad", [(6, 200, 0), (6, 200, 3), (5, 1032, 8), (3, 333, 1), (620, 1032, 8)])
def test_forward_forms(nv, stream, post, gate, m, n, pad):
    """Every combination of what may be absent, both stream types, rows of a wider buffer."""
    d = inputs(m, n, stream, post, gate, pad=pad)
    x_out, h = nv.block_norm(d["x"], d["w_pre"], y=d["y"], w_post=d["w_post"], gate=d["gate"], residual_scale=1.3, eps=EPS,
                             weight_offset=1.0)
    r_ref, h_ref = block.block_norm(f64(d["x"]), f64(d["w_pre"]), f64(d["y"]), f64(d["w_post"]), f64(d["gate"]), 1.3, EPS, 1.0)
    tr, th = forward_terms(d, 1.3, 1.0)
    if post is None:
        assert x_out is d["x"]
    check(x_out, r_ref, BF16 if stream == torch.bfloat16 else 2.0 ** -23, tr, "x_out")
    check(h, h_ref, BF16, th, "h")


def test_forward_in_place_and_without_the_second_norm(nv):
    d = inputs(40, 1024)
    want, none = nv.block_norm(d["x"], None, y=d["y"], w_post=d["w_post"])
    assert none is None
    both, h = nv.block_norm(d["x"], d["w_pre"], y=d["y"], w_post=d["w_post"])
    assert torch.equal(both, want)
    x = d["x"].clone()
    out, h2 = nv.block_norm(x, d["w_pre"], y=d["y"], w_post=d["w_post"], x_out=x)
    assert out is x and torch.equal(x, want) and torch.equal(h, h2)


def test_forward_in_place_with_rows_copied_ahead(nv):
    d = inputs(1300, 2048, gate="token")
    kw = dict(y=d["y"], w_post=d["w_post"], gate=d["gate"])
    want, h = nv.block_norm(d["x"], d["w_pre"], **kw)
    x = d["x"].clone()
    out, h2 = nv.block_norm(x, d["w_pre"], x_out=x, **kw)
    assert out is x and torch.equal(x, want) and torch.equal(h, h2)
    none, h3 = nv.block_norm(want, d["w_pre"])
    assert none is want and h3.shape == h.shape


def test_zero_rows_and_special_values(nv):
    d = inputs(4, 64)
    for t in ("x", "y"):
        d[t] = torch.zeros_like(d[t])
    x_out, h = nv.block_norm(d["x"], d["w_pre"], y=d["y"], w_post=d["w_post"], gate=d["gate"])
    assert not x_out.any() and not h.any()                       # 0 * rsqrt(eps), not 0 / 0
    x = torch.randn(3, 64).to(torch.bfloat16).cuda()
    x[1, 5] = float("nan")
    _, h = nv.block_norm(x, d["w_pre"])
    assert torch.isnan(h[1]).all() and not torch.isnan(h[0]).any() and not torch.isnan(h[2]).any()
    x_out, h = nv.block_norm(x[:0], d["w_pre"], y=x[:0])
    assert x_out.shape == (0, 64) and h.shape == (0, 64)


@pytest.mark.parametrize("m,n", [(1, 16), (1, 7168), (3, 48), (130, 1024), (128, 4096), (5, 496), (300, 528), (2, 20480), (610, 528),
                                 (650, 2080), (640, 4096)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_quantized_output_equals_the_two_calls(nv, m, n, stream):
    d = inputs(m, n, stream, gate="token")
    kw = dict(y=d["y"], w_post=d["w_post"], gate=d["gate"], residual_scale=0.5)
    x_out, h = nv.block_norm(d["x"], d["w_pre"], **kw)
    gs = (2688.0 / h.float().abs().max()).reshape(1)
    q_ref, sf_ref = nv.nvfp4_quantize(h, gs)
    sf = torch.full_like(sf_ref, 0xAA)
    x2, q, sf = nv.block_norm_quantize(d["x"], d["w_pre"], gs, sf=sf, flags=nv.FLAG_PDL, **kw)
    assert torch.equal(x_out, x2) and torch.equal(q, q_ref) and torch.equal(sf, sf_ref)
    qo, so = oquant.nvfp4_quantize(h.cpu(), np.float32(gs.item()))
    assert np.array_equal(q.cpu().numpy(), qo) and np.array_equal(sf.cpu().numpy(), so)


def backward_terms(d, r, scale, offset):
    """Magnitudes that enter dx, dy and the sums over rows."""
    ab = lambda t: np.abs(f64(t))  # noqa: E731
    rstd = 1.0 / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + EPS)
    xn = np.abs(r * rstd)
    t = {}
    g = ab(d["dr"]) if d["dr"] is not None else np.zeros_like(r)
    if d["w_pre"] is not None:
        dd = ab(d["dh"]) * np.abs(offset + f64(d["w_pre"]))
        g = g + rstd * (dd + xn * np.mean(dd * xn, axis=1, keepdims=True))
        t["dw_pre"] = np.sum(ab(d["dh"]) * xn, axis=0)
    t["dx"] = g
    if d["y"] is not None:
        y = f64(d["y"])
        ry = 1.0 / np.sqrt(np.mean(y * y, axis=1, keepdims=True) + EPS) if d["w_post"] is not None else 1.0
        w = np.abs(offset + f64(d["w_post"])) if d["w_post"] is not None else 1.0
        yn, b = np.abs(y) * ry, abs(scale) * g
        if d["gate"] is not None:
            t["dgate"] = b * yn * w
            if d["gate"].dim() == 1:
                t["dgate"] = t["dgate"].sum(axis=0)
            b = b * ab(d["gate"])
        t["dw_post"] = np.sum(b * yn, axis=0)
        e = b * w
        t["dy"] = ry * (e + yn * np.mean(e * yn, axis=1, keepdims=True)) if d["w_post"] is not None else b
    return t


def check_backward(nv, d, scale, offset, **kw):
    stream = d["x"].dtype
    got = nv.block_norm_backward(d["dh"] if d["w_pre"] is not None else None, d["dr"], d["x"], d["w_pre"], y=d["y"],
                                 w_post=d["w_post"], gate=d["gate"], residual_scale=scale, eps=EPS, weight_offset=offset, **kw)
    ref = block.block_norm_backward(f64(d["dh"]) if d["w_pre"] is not None else None, f64(d["dr"]), f64(d["x"]),
                                    f64(d["w_pre"]), f64(d["y"]), f64(d["w_post"]), f64(d["gate"]), scale, EPS, offset)
    t = backward_terms(d, f64(d["x"]), scale, offset)
    for name, a, b in zip(("dx", "dy", "dw_pre", "dw_post", "dgate"), got, ref):
        assert (a is None) == (b is None), name
        if a is not None:
            assert a.shape == b.shape
            rounding = 2.0 ** -23 if a.dtype == torch.float32 else BF16
            check(a, b, rounding, 2 * t[name], name)
    assert got[0].dtype == stream
    return got


@pytest.mark.parametrize("m,n", SHAPES)
def test_backward(nv, m, n):
    d = inputs(m, n)
    check_backward(nv, d, 0.7, 0.0)


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("post,gate", [(True, "none"), (True, "channel"), (True, "token"), (False, "none"), (False, "channel"),
                                       (False, "token"), (None, "none")])
@pytest.mark.parametrize("m,n,pad", [(6, 200, 0), (700, 200, 3), (5, 1032, 8), (3, 333, 1), (620, 1032, 8)])
def test_backward_forms(nv, stream, post, gate, m, n, pad):
    d = inputs(m, n, stream, post, gate, pad=pad)
    check_backward(nv, d, 1.3, 1.0)
    d["dr"] = None
    check_backward(nv, d, 1.3, 1.0)


# Rows of single channels (n no multiple of 8, or a wider buffer that breaks the alignment) over every block size,
# and blocks of several to an SM; 4097 to 6144 channels also aligned with few rows.
PLAIN = [(1500, 523, 0), (700, 723, 0), (1300, 1025, 0), (400, 2561, 0), (160, 4097, 0), (3, 6001, 0), (3, 5000, 0), (160, 6144, 3),
         (5, 7169, 0), (2, 8200, 1), (160, 12289, 0), (2, 16385, 0), (1, 32767, 0)]


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,pad", PLAIN)
def test_single_channels(nv, m, n, pad, stream):
    d = inputs(m, n, stream, pad=pad)
    x_out, h = nv.block_norm(d["x"], d["w_pre"], y=d["y"], w_post=d["w_post"], gate=d["gate"], residual_scale=0.7, eps=EPS)
    r_ref, h_ref = block.block_norm(f64(d["x"]), f64(d["w_pre"]), f64(d["y"]), f64(d["w_post"]), f64(d["gate"]), 0.7, EPS)
    tr, th = forward_terms(d, 0.7, 0.0)
    check(x_out, r_ref, BF16 if stream == torch.bfloat16 else 2.0 ** -23, tr, "x_out")
    check(h, h_ref, BF16, th, "h")
    check_backward(nv, d, 0.7, 0.0)


@pytest.mark.parametrize("post,gate", [(True, "token"), (False, "none"), (None, "none")])
@pytest.mark.parametrize("m,n", [(3, 5001), (3, 5000), (2, 7001), (2, 9001), (2, 20001)])
def test_absent_operands_of_wide_rows(nv, m, n, post, gate):
    """What is not there reads as zero in every block size, whether loaded ahead or not."""
    d = inputs(m, n, torch.bfloat16, post, gate)
    check_backward(nv, d, 1.3, 1.0)
    d["dr"] = None
    check_backward(nv, d, 1.3, 1.0)
    if post is not None:
        d["w_pre"] = None
        check_backward(nv, d, 0.9, 0.0)


def test_backward_without_the_second_norm_and_without_rows(nv):
    d = inputs(33, 512, gate="token")
    d["w_pre"] = None
    check_backward(nv, d, 0.9, 0.0)
    e = inputs(4, 96)
    z = {k: (v[:0] if v is not None and v.dim() == 2 else v) for k, v in e.items()}
    dx, dy, dw_pre, dw_post, dgate = nv.block_norm_backward(z["dh"], z["dr"], z["x"], z["w_pre"], y=z["y"], w_post=z["w_post"],
                                                            gate=z["gate"])
    assert dx.shape == dy.shape == (0, 96)
    assert not dw_pre.any() and not dw_post.any() and not dgate.any()


def test_backward_is_bit_reproducible(nv):
    d = inputs(700, 4096)
    one = check_backward(nv, d, 1.0, 0.0)
    for _ in range(3):
        two = nv.block_norm_backward(d["dh"], d["dr"], d["x"], d["w_pre"], y=d["y"], w_post=d["w_post"], gate=d["gate"], eps=EPS)
        for a, b in zip(one, two):
            assert torch.equal(a, b)


@pytest.mark.parametrize("gate", ["channel", "token"])
def test_backward_against_differences(nv, gate):
    """The GPU's gradients along a random direction against central differences of the fp64 forward
    pass.  r does not depend on rounding here: the backward pass is given the fp64 stream rounded to
    fp32, whose error (2^-24 of a value) is far below the gradients' own bf16 rounding.  A directional
    derivative is a sum of gradient * direction: the bf16 gradients are off by at most 2^-8 of each
    term, the others by FP32 of theirs; the differences (step 1e-5, third derivatives of order one)
    by 1e-8 of the terms."""
    m, n = 5, 136
    d = inputs(m, n, torch.float32, True, gate, seed=3)
    v = {k: f64(d[k]) for k in ("x", "y", "w_post", "w_pre", "gate")}
    f = lambda a: block.block_norm(a["x"], a["w_pre"], a["y"], a["w_post"], a["gate"], 0.8, EPS, 0.0)  # noqa: E731
    r, _ = f(v)
    stored = torch.from_numpy(r).float().cuda()
    got = nv.block_norm_backward(d["dh"], d["dr"], stored, d["w_pre"], y=d["y"], w_post=d["w_post"], gate=d["gate"],
                                 residual_scale=0.8, eps=EPS)
    got = dict(zip(("x", "y", "w_pre", "w_post", "gate"), got))
    rng = np.random.default_rng(5)
    for name in v:
        dv = rng.standard_normal(v[name].shape)
        loss = []
        for s in (1e-5, -1e-5):
            a = dict(v)
            a[name] = v[name] + s * dv
            rr, hh = f(a)
            loss.append(np.sum(rr * f64(d["dr"])) + np.sum(hh * f64(d["dh"])))
        want = (loss[0] - loss[1]) / 2e-5
        gr = f64(got[name])
        tol = (BF16 if got[name].dtype == torch.bfloat16 else 2.0 ** -15) * np.sum(np.abs(gr * dv)) + 1e-6
        assert abs(np.sum(gr * dv) - want) <= tol, name


def test_another_stream(nv):
    """Inputs made on one stream, the call on another that waits for them."""
    d = inputs(64, 2048)
    want = nv.block_norm(d["x"], d["w_pre"], y=d["y"], w_post=d["w_post"])[1]
    g_want = nv.block_norm_backward(d["dh"], d["dr"], d["x"], d["w_pre"], y=d["y"], w_post=d["w_post"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        h = nv.block_norm(d["x"], d["w_pre"], y=d["y"], w_post=d["w_post"])[1]
        g = nv.block_norm_backward(d["dh"], d["dr"], d["x"], d["w_pre"], y=d["y"], w_post=d["w_post"])
    s.synchronize()
    assert torch.equal(h, want) and all(a is b or torch.equal(a, b) for a, b in zip(g, g_want))


def test_broadcast_inputs(nv):
    """Rows expanded from one row are read as they are; the gradients come for every row."""
    m, n = 7, 264
    d = inputs(m, n, gate="token")
    for k in ("x", "y", "gate", "dh", "dr"):
        d[k] = d[k][:1].expand(m, n)
    full = {k: (v.contiguous() if v is not None else None) for k, v in d.items()}
    for a, b in zip(nv.block_norm(d["x"], d["w_pre"], y=d["y"], w_post=d["w_post"], gate=d["gate"]),
                    nv.block_norm(full["x"], full["w_pre"], y=full["y"], w_post=full["w_post"], gate=full["gate"])):
        assert torch.equal(a, b)
    got = check_backward(nv, d, 0.7, 0.0)
    want = check_backward(nv, full, 0.7, 0.0)
    assert got[4].shape == (m, n)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(nv):
    """Rows whose element offsets pass 2^31 (three rows, 2^30 + 8 elements apart), in and out."""
    m, n, ld = 3, 1032, (1 << 30) + 8
    d = inputs(m, n, gate="token")
    buf = torch.empty(2 * ld + n, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((m, n), (ld, 1))
    kw = dict(y=d["y"], w_post=d["w_post"], gate=d["gate"])
    want, h = nv.block_norm(d["x"], d["w_pre"], **kw)
    for k in ("x", "y", "gate"):
        far.copy_(d[k])
        got = nv.block_norm(**{**dict(x=d["x"], w_pre=d["w_pre"]), **kw, k: far})
        assert torch.equal(got[0], want) and torch.equal(got[1], h)
    nv.block_norm(d["x"], d["w_pre"], **kw, h=far)
    assert torch.equal(far, h)
    nv.block_norm(d["x"], d["w_pre"], **kw, x_out=far)
    assert torch.equal(far, want)
    g = nv.block_norm_backward(d["dh"], d["dr"], d["x"], d["w_pre"], **kw)
    far.copy_(d["dh"])
    for a, b in zip(g, nv.block_norm_backward(far, d["dr"], d["x"], d["w_pre"], **kw)):
        assert torch.equal(a, b)


def test_rows_copied_ahead_past_32_bits(nv):
    """More elements than 2^31 in rows that are brought ahead through shared memory."""
    m, n = 262200, 8192
    x = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(40, n, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    x[-40:] = last
    _, h = nv.block_norm(x, w)
    assert torch.equal(h[-40:], nv.block_norm(torch.cat([last] * 20), w)[1][:40])
    assert not h[:40].any()
    dx = nv.block_norm_backward(h, None, x, w)[0]
    want = nv.block_norm_backward(torch.cat([h[-40:]] * 20), None, torch.cat([last] * 20), w)[0][:40]
    assert torch.equal(dx[-40:], want)
