"""e4m3 quantisation with a scale per block of 128 and the products of such matrices on the GPU: the
quantisers bit for bit against the oracle, the products against fp64 within the bound of their sums."""
import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8
from oracle.formats import e4m3_decode

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_bf16_gb300 as m
    torch.cuda.set_device(0)
    yield m
    m.check_status()


def rng(seed):
    return np.random.default_rng(seed)


def matrix(seed, m, k, dtype="bf16", scale=1.0):
    """Values over several binades, whole zero blocks among them."""
    r = rng(seed)
    x = r.standard_normal((m, k)) * np.exp2(r.integers(-6, 7, (m, 1))) * scale
    x[:, :: max(1, k // 4)] *= 20.0
    x[r.random((m, k)) < 0.05] = 0.0
    if k >= 256 and m > 1:
        x[m // 2, 128:256] = 0.0
    return torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype]).cuda()


def host(t):
    return t.view(torch.uint8).cpu().numpy() if t.dtype == torch.float8_e4m3fn else t.float().cpu().numpy()


def same(got, want):
    for g, w in zip(got, want):
        g = host(g)
        assert g.shape == w.shape
        assert np.array_equal(g, w, equal_nan=g.dtype.kind == "f"), np.argwhere(~((g == w) | ((g != g) & (w != w))))[:4]


def test_quantize_nothing(nv):
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    q, sf, qt, sft = nv.fp8_quantize(x, transpose=True)
    assert q.shape == (0, 256) and sf.shape == (2, 0) and qt.shape == (256, 0) and sft.shape == (0, 256)
    assert nv.fp8_quantize(x)[0].shape == (0, 256)


SIZES = [(1, 16), (1, 7168), (3, 48), (31, 128), (33, 2080), (128, 256), (129, 144), (300, 1040), (515, 640)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,k", SIZES)
def test_quantize_rows_and_columns(nv, m, k, dtype):
    x = matrix(m * k, m, k, dtype)
    xn = x.float().cpu().numpy()
    rows, cols = ofp8.quantize_rows(xn), ofp8.quantize_columns(xn)
    same(nv.fp8_quantize(x), rows)
    same(nv.fp8_quantize(x, transpose=True), rows + cols)
    same(nv.fp8_quantize(x, rows=False, transpose=True), cols)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,k", [(3000, 1040), (2100, 2048)])
def test_quantize_many_rows(nv, m, k, dtype):
    """Enough blocks for the variants that take several in turn."""
    x = matrix(5, m, k, dtype)
    xn = x.float().cpu().numpy()
    same(nv.fp8_quantize(x), ofp8.quantize_rows(xn))
    same(nv.fp8_quantize(x, transpose=True), ofp8.quantize_rows(xn) + ofp8.quantize_columns(xn))


def test_quantize_every_bf16_value(nv):
    """Every finite bf16 magnitude in one block with each of several largest values: all roundings of the codes."""
    bits = np.arange(0x7F80, dtype=np.uint32)
    vals = (bits << 16).view(np.float32)
    rows = []
    for top in (1.0, 3.0, 448.0, 1.9921875, 2.0 ** -90, 2.0 ** -101, 3.3895314e38):
        v = vals[vals <= np.float32(top)][-126 * 30:]
        v = np.pad(v, (0, -len(v) % 126)).reshape(-1, 126)
        signed = v * np.where(np.arange(126) % 2, -1, 1).astype(np.float32)
        rows.append(np.concatenate([signed, np.full((len(v), 1), top, np.float32), np.zeros((len(v), 1), np.float32)], 1))
    x = torch.from_numpy(np.concatenate(rows)).to(torch.bfloat16).cuda()
    xn = x.float().cpu().numpy()
    same(nv.fp8_quantize(x, transpose=True), ofp8.quantize_rows(xn) + ofp8.quantize_columns(xn))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_rows_of_a_wider_buffer_and_by_index(nv, dtype):
    unit = 8 if dtype == "bf16" else 4
    wide = matrix(7, 70, 512 + unit, dtype)
    x = wide[:, unit: unit + 400]                     # rows that start on 16 bytes, not on 32
    xn = x.float().cpu().numpy()
    want = ofp8.quantize_rows(xn) + ofp8.quantize_columns(xn)
    same(nv.fp8_quantize(x, transpose=True), want)
    same(nv.fp8_quantize(x), want[:2])
    idx = rng(3).integers(0, 70, 201).astype(np.int32)
    src = torch.from_numpy(idx).cuda()
    want = ofp8.quantize_rows(xn[idx]) + ofp8.quantize_columns(xn[idx])
    same(nv.fp8_quantize(x, src_rows=src, transpose=True), want)
    same(nv.fp8_quantize(x, src_rows=src), want[:2])
    same(nv.fp8_quantize(x, src_rows=src, rows=False, transpose=True), want[2:])


@pytest.mark.parametrize("m", [3, 200])
def test_quantize_non_finite_and_tiny(nv, m):
    """A block with an infinity or a NaN gives no finite value, others are untouched; blocks under 2^-100 round
    as their scale's floor says."""
    x = matrix(11, m, 512, "f32").clone()
    x[0, 5], x[1, 130], x[2, 300] = float("inf"), float("nan"), float("-inf")
    x[1, 384:] = 2.0 ** -110
    x[0, 384:] = 2.0 ** -140
    xn = x.cpu().numpy()
    q, sf, qt, sft = nv.fp8_quantize(x, transpose=True)
    # the codes of a block that holds one are given by the same steps, but for the sign of NaN
    for got, want in zip((q, sf, qt, sft), ofp8.quantize_rows(xn) + ofp8.quantize_columns(xn)):
        g = host(got)
        if g.dtype == np.uint8:
            assert np.array_equal(e4m3_decode(g), e4m3_decode(want), equal_nan=True)
        else:
            assert np.array_equal(g, want, equal_nan=True)
    with np.errstate(invalid="ignore"):
        v = e4m3_decode(host(q)) * np.repeat(host(sf).astype(np.float64).T, 128, 1)
    assert not np.isfinite(v[0, :128]).any() and not np.isfinite(v[1, 128:256]).any() and not np.isfinite(v[2, 256:384]).any()
    assert np.isfinite(v[0, 128:]).all() and np.isfinite(v[2, :256]).all()


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts", [[1], [0], [128], [0, 5, 0, 127, 128, 129, 0], [300, 0, 1, 260], list(range(40)), [3] * 70])
def test_quantize_experts(nv, counts, dtype):
    ro = offsets_of(counts)
    k = 400
    rows = int(ro[-1])
    x = matrix(13, 50, k, dtype)
    idx = rng(5).integers(0, 50, rows).astype(np.int32)
    xn = x.float().cpu().numpy()[idx]
    src, off = torch.from_numpy(idx).cuda(), torch.from_numpy(ro).cuda()
    q, sf, qt, sft = nv.fp8_quantize(x, src_rows=src, row_offsets=off, transpose=True)
    want = ofp8.quantize_columns(xn, ro)
    same((qt, sft), want)
    if rows:
        same((q, sf), ofp8.quantize_rows(xn))
    same(nv.fp8_quantize(x, src_rows=src, row_offsets=off, rows=False, transpose=True), want)
    nv.check_status()


def test_quantize_rows_past_the_last_expert_stay(nv):
    ro = np.array([0, 100, 130], np.int64)
    x = matrix(17, 200, 256)
    xn = x.float().cpu().numpy()
    q = torch.full((200, 256), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sf = torch.full((2, 200), -7.0, device="cuda")
    _, _, qt, sft = nv.fp8_quantize(x, row_offsets=torch.from_numpy(ro).cuda(), transpose=True, q=q, sf=sf)
    wq, ws = ofp8.quantize_rows(xn)
    assert np.array_equal(host(q)[:130], wq[:130]) and (host(q)[130:] == 0x55).all()
    assert np.array_equal(host(sf)[:, :130], ws[:, :130]) and (host(sf)[:, 130:] == -7.0).all()
    same((qt, sft), ofp8.quantize_columns(xn, ro))


def test_quantize_reports_bad_indices_and_offsets(nv):
    x = matrix(19, 10, 128)
    src = torch.tensor([0, 10, -1, 3], dtype=torch.int32, device="cuda")
    xn = x.float().cpu().numpy()
    want = xn[[0, 0, 0, 3]]
    want[1:3] = 0
    for transpose in (False, True):
        got = nv.fp8_quantize(x, src_rows=src, transpose=transpose)
        same(got, ofp8.quantize_rows(want) + (ofp8.quantize_columns(want) if transpose else ()))
        with pytest.raises(nv.NVFP4Error):
            nv.check_status()
    for bad in ([1, 5, 10], [0, 7, 5], [0, 4, 11], [0, -3, 10]):
        qt, sft = nv.fp8_quantize(x, row_offsets=torch.tensor(bad, device="cuda"), rows=False, transpose=True)
        assert (host(qt) == 0).all()
        with pytest.raises(nv.NVFP4Error):
            nv.check_status()
    nv.check_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(16, 16), (128, 128), (144, 400), (784, 1040), (1008, 2080)])
def test_quantize_weight(nv, n, k, dtype):
    w = matrix(n + k, n, k, dtype, 0.02)
    q, s = ofp8.quantize_blocks(w.float().cpu().numpy())
    same(nv.fp8_quantize_weight(w), (q, s))
    same(nv.fp8_quantize_weight(w, transpose=True), (q, s, np.ascontiguousarray(q.T), np.ascontiguousarray(s.T)))
    assert n == 16 or torch.equal(nv.fp8_quantize_weight(w[: n - 3])[0].view(torch.uint8),
                                  nv.fp8_quantize_weight(w[: n - 3].clone())[0].view(torch.uint8))


def test_quantize_weights_of_experts(nv):
    w = torch.stack([matrix(i, 208, 272, "f32", 0.02 * (i + 1)) for i in range(5)])
    got = nv.fp8_quantize_weight(w, transpose=True)
    for e in range(5):
        q, s = ofp8.quantize_blocks(w[e].cpu().numpy())
        same([g[e] for g in got], (q, s, np.ascontiguousarray(q.T), np.ascontiguousarray(s.T)))
    odd = w[:, :201].contiguous()                     # rows that fill no block, no transpose of them
    got = nv.fp8_quantize_weight(odd)
    for e in range(5):
        same([g[e] for g in got], ofp8.quantize_blocks(odd[e].cpu().numpy()))


# ------------------------------------------------------------------ products
def codes(seed, shape):
    """Codes of all magnitudes, both signs, no NaN."""
    c = rng(seed).integers(0, 256, shape).astype(np.uint8)
    c[(c & 0x7F) == 0x7F] = 0x30
    return torch.from_numpy(c).cuda().view(torch.float8_e4m3fn)


def scales(seed, shape):
    return torch.from_numpy(np.exp(rng(seed).standard_normal(shape)).astype(np.float32)).cuda()


def rows64(q, s):
    return q.double() * s.double().t().repeat_interleave(128, 1)[:, : q.shape[1]]


def blocks64(q, s):
    n, k = q.shape
    return q.double() * s.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]


def check_product(d, a, b, k, old=None):
    """|D - R| within half a step of D's type and the slack of the sums; accumulated: one more fp32 rounding."""
    r, size = a @ b.t(), a.abs() @ b.abs().t()
    tol = ofp8.product_slack(k) * size
    if old is not None:
        r = r + old.double()
        tol = tol + 2.0 ** -24 * r.abs()
    tol = tol + torch.finfo(d.dtype).eps / 2 * (r.abs() + tol)
    err = (d.double() - r).abs()
    assert torch.isfinite(d).all() and (err <= tol).all(), (float((err - tol).max()), int((err > tol).sum()), d.shape)


PRODUCTS = [(1, 1, 16), (1, 128, 128), (1, 4096, 7168), (2, 1001, 2080), (16, 256, 1024), (17, 384, 400), (32, 640, 256),
            (33, 130, 1040), (64, 784, 2048), (65, 200, 272), (100, 1000, 2080), (128, 1536, 512), (129, 257, 144), (256, 256, 256),
            (300, 1001, 2080), (385, 513, 1168), (1000, 3000, 640), (2048, 1536, 2048)]


@pytest.mark.parametrize("block_b", [128, 1])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_gemm(nv, m, n, k, out, block_b):
    kb = -(-k // 128)
    a, sa, b = codes(m, (m, k)), scales(m + 1, (kb, m)), codes(n, (n, k))
    sb = scales(n + 1, (-(-n // 128), kb) if block_b == 128 else (kb, n))
    d = torch.full((m + 1, n), -3.0, dtype=TYPES[out], device="cuda")
    nv.fp8_gemm(a, sa, b, sb, block_b=block_b, d=d[:m])
    va, vb = rows64(a, sa), blocks64(b, sb) if block_b == 128 else rows64(b, sb)
    check_product(d[:m], va, vb, k)
    assert (d[m] == -3.0).all()
    if out == "f32":
        old = d[:m].clone()
        nv.fp8_gemm(a, sa, b, sb, block_b=block_b, d=d[:m], accumulate=True)
        check_product(d[:m], va, vb, k, old)
    nv.check_status()


@pytest.mark.parametrize("m,n,k", [(1, 256, 512), (40, 256, 512), (300, 512, 512)])
def test_gemm_is_reproducible_and_pdl_changes_nothing(nv, m, n, k):
    x = matrix(1, m, k)
    w = matrix(2, n, k, "f32", 0.02)
    q, sf = nv.fp8_quantize(x)
    b, sb = nv.fp8_quantize_weight(w)
    want = nv.fp8_gemm(q, sf, b, sb)
    for _ in range(5):
        q2, sf2 = nv.fp8_quantize(x, flags=nv.FLAG_PDL)
        assert torch.equal(nv.fp8_gemm(q2, sf2, b, sb, flags=nv.FLAG_PDL), want)


def test_gemm_nan_stays_in_its_row_and_column(nv):
    for m in (8, 300):
        a, sa = codes(1, (m, 256)), scales(2, (2, m))
        b, sb = codes(3, (140, 256)), scales(4, (2, 2))
        a.view(torch.uint8)[5, 130] = 0x7F
        sa[0, 2] = float("inf")
        b.view(torch.uint8)[7, 3] = 0xFF
        d = nv.fp8_gemm(a, sa, b, sb)
        bad = torch.zeros(m, 140, dtype=torch.bool, device="cuda")
        bad[5], bad[2], bad[:, 7] = True, True, True
        assert torch.equal(~torch.isfinite(d), bad)


def experts(seed, counts, k, n):
    ro = offsets_of(counts)
    t, e, kb = int(ro[-1]), len(counts), -(-k // 128)
    return (torch.from_numpy(ro).cuda(), ro, codes(seed, (t, k)), scales(seed + 1, (kb, t)), codes(seed + 2, (e, n, k)),
            scales(seed + 3, (e, -(-n // 128), kb)))


COUNTS = [[1], [5, 0, 3], [0, 0, 16, 1], [16] * 9, [17, 0, 33, 64, 1, 40], [128, 0, 129, 1, 255, 256], [300, 700, 0, 50], [0] * 30 + [500] + [0] * 33,
          [2] * 100, list(range(0, 90, 3)), [1] * 1024]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(256, 256), (200, 400), (129, 1040)])
@pytest.mark.parametrize("counts", COUNTS, ids=range(len(COUNTS)))
def test_grouped(nv, counts, n, k, out):
    off, ro, a, sa, b, sb = experts(21, counts, k, n)
    t = int(ro[-1])
    d = torch.full((t + 3, n), -3.0, dtype=TYPES[out], device="cuda")
    nv.fp8_grouped_gemm(a, sa, off, b, sb, d=d[:t])
    va = rows64(a, sa)
    for e in range(len(counts)):
        if counts[e]:
            check_product(d[ro[e]: ro[e + 1]], va[ro[e]: ro[e + 1]], blocks64(b[e], sb[e]), k)
    assert (d[t:] == -3.0).all()
    nv.check_status()


@pytest.mark.parametrize("mean", [1, 300])
def test_grouped_rows_past_the_last_expert_stay(nv, mean):
    counts = [mean, 0, 2 * mean]
    off, ro, a, sa, b, sb = experts(23, counts + [40], 256, 200)
    off = off[:4].contiguous()
    t = a.shape[0]
    d = torch.full((t, 200), -3.0, dtype=torch.bfloat16, device="cuda")
    nv.fp8_grouped_gemm(a, sa, off, b[:3].contiguous(), sb[:3].contiguous(), d=d)
    va = rows64(a, sa)
    for e in (0, 2):
        check_product(d[ro[e]: ro[e + 1]], va[ro[e]: ro[e + 1]], blocks64(b[e], sb[e]), 256)
    assert (d[ro[3]:] == -3.0).all()
    nv.check_status()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(256, 256), (200, 400), (784, 1040), (129, 33)])
@pytest.mark.parametrize("counts", [[1], [0], [0, 128, 0], [5, 0, 129, 1, 300], [127, 128, 129], [260] * 5, [2] * 40])
def test_weight_grad(nv, counts, n, k, out):
    ro = offsets_of(counts)
    t, e = int(ro[-1]), len(counts)
    place, p = ofp8.padded_place(ro, t)
    a, b = codes(31, (n, p)), codes(32, (k, p))
    pad = torch.ones(p, dtype=torch.bool, device="cuda")
    pad[torch.from_numpy(place).cuda()] = False
    # the quantiser leaves zeros between the experts; what lies behind the last one is never read
    last = sum(-(-c // 128) * 128 for c in counts)
    pad[last:] = False
    a.view(torch.uint8)[:, pad] = 0
    b.view(torch.uint8)[:, pad] = 0
    a.view(torch.uint8)[:, last:] = 0x7F
    b.view(torch.uint8)[:, last:] = 0x7F
    sa, sb = scales(33, (p // 128, n)), scales(34, (p // 128, k))
    off = torch.from_numpy(ro).cuda()
    d = nv.fp8_grouped_weight_grad(a, sa, b, sb, off, out_dtype=TYPES[out])
    old = d.clone()
    if out == "f32":
        nv.fp8_grouped_weight_grad(a, sa, b, sb, off, d=d, accumulate=True)
    va, vb = rows64(a, sa), rows64(b, sb)
    at = 0
    for i in range(e):
        c = counts[i]
        if c == 0:
            assert (d[i] == 0).all()
        else:
            check_product(old[i], va[:, at: at + c], vb[:, at: at + c], c)
            if out == "f32":
                check_product(d[i], va[:, at: at + c], vb[:, at: at + c], c, old[i])
        at += -(-c // 128) * 128
    nv.check_status()


def test_grouped_malformed_offsets_do_nothing(nv):
    off, ro, a, sa, b, sb = experts(41, [10, 20, 30], 256, 128)
    pa, pb = codes(1, (64, 512)), codes(2, (128, 512))
    for bad in ([1, 10, 30, 60], [0, 30, 10, 60], [0, 10, 30, 61], [0, -5, 30, 60], [0, 10, 30, 1 << 40]):
        o = torch.tensor(bad, device="cuda")
        d = torch.full((60, 128), -3.0, dtype=torch.bfloat16, device="cuda")
        nv.fp8_grouped_gemm(a, sa, o, b, sb, d=d)
        with pytest.raises(nv.NVFP4Error):
            nv.check_status()
        assert (d == -3.0).all()
    for bad in ([1, 10, 30, 60], [0, 30, 10, 60], [0, 129, 258, 387], [0, -5, 30, 60], [0, 10, 30, 1 << 40]):
        o = torch.tensor(bad, device="cuda")
        g = torch.full((3, 64, 128), -3.0, device="cuda")
        nv.fp8_grouped_weight_grad(pa, scales(3, (4, 64)), pb, scales(4, (4, 128)), o, d=g)
        with pytest.raises(nv.NVFP4Error):
            nv.check_status()
        assert (g == -3.0).all()


@pytest.mark.parametrize("m", [4, 300])
def test_a_wait_that_runs_out_is_reported(nv, m):
    """The copy of the first stage is left out: the bounded waits give up, the status says so, and the next call works."""
    a, sa, b, sb = codes(1, (m, 512)), scales(2, (4, m)), codes(3, (256, 512)), scales(4, (2, 4))
    nv.fp8_gemm(a, sa, b, sb, flags=nv.FLAG_DEBUG_TIMEOUT | nv.FLAG_DEBUG_SKIP_FIRST_LOAD)
    with pytest.raises(nv.NVFP4Error) as e:
        nv.check_status()
    assert e.value.code == 6
    check_product(nv.fp8_gemm(a, sa, b, sb), rows64(a, sa), blocks64(b, sb), 512)
    nv.check_status()


def test_on_another_stream_and_in_a_graph(nv):
    """Outputs are made for the launch stream; a captured chain replays on new inputs."""
    m, n, k = 70, 256, 384
    x, w = matrix(51, m, k), matrix(52, n, k, "f32", 0.02)
    b, sb = nv.fp8_quantize_weight(w)
    want = nv.fp8_gemm(*nv.fp8_quantize(x), b, sb)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q, sf = nv.fp8_quantize(x, stream=s)
    d = nv.fp8_gemm(q, sf, b, sb, stream=s)
    s.synchronize()
    assert torch.equal(d, want)
    buf = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = nv.fp8_gemm(*nv.fp8_quantize(buf), b, sb)
    buf.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
