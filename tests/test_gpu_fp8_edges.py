"""The 8-bit products at their edges on the GPU: every choice of tiles, offsets past 32 bits, several streams at once,
captured chains, and an expert layer forward and backward, each step against fp64 of the operands it was given."""
import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_bf16_gb300 as m
    torch.cuda.set_device(0)
    yield m
    m.check_status()


def codes(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    c[(c & 0x7F) == 0x7F] = 0x30
    return c.view(torch.float8_e4m3fn)


def scales(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.exp(torch.randn(*shape, generator=g, device="cuda"))


def rows64(q, s):
    return q.double() * s.double().t().repeat_interleave(128, 1)[:, : q.shape[1]]


def blocks64(q, s):
    n, k = q.shape[-2:]
    return q.double() * s.double().repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]


def within(d, a, b, k):
    """Half a step of D's type and the slack of the sums (see ofp8.product_slack)."""
    r = a @ b.t()
    tol = ofp8.product_slack(k) * (a.abs() @ b.abs().t())
    tol = tol + torch.finfo(d.dtype).eps / 2 * (r.abs() + tol)
    err = (d.double() - r).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("block_b", [128, 1])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("m,n,k", [(140, 1000, 256), (200, 2000, 256), (256, 4096, 4096), (300, 1008, 2080), (520, 4096, 1040), (1030, 2040, 1024),
                                   (1500, 3080, 640), (2100, 4100, 400), (129, 8, 7168), (4100, 264, 128), (150, 333, 7168), (5000, 16, 16)])
def test_every_choice_of_tiles(nv, m, n, k, out, block_b):
    """Sizes of more than 128 tokens at which each of the five kinds of tiles is the cheapest, rows that leave as bulk
    copies and rows that do not, ends inside a tile, a copy's box and a row's sixteen bytes."""
    kb = -(-k // 128)
    a, sa, b = codes(m, m, k), scales(1, kb, m), codes(n, n, k)
    sb = scales(2, -(-n // 128), kb) if block_b == 128 else scales(2, kb, n)
    d = torch.full((m + 2, n), -3.0, dtype=out, device="cuda")
    nv.fp8_gemm(a, sa, b, sb, block_b=block_b, d=d[:m])
    within(d[:m], rows64(a, sa), blocks64(b, sb) if block_b == 128 else rows64(b, sb), k)
    assert bool((d[m:] == -3.0).all())
    nv.check_status()


def test_results_past_32_bit_offsets(nv):
    """A result and a quantised matrix of more than 2^31 elements: their ends."""
    m, n, k = 66000, 33000, 128
    a, sa, b, sb = codes(1, m, k), scales(2, 1, m), codes(3, n, k), scales(4, 258, 1)
    d = nv.fp8_gemm(a, sa, b, sb)
    for r in (0, 131, m - 129, m - 1):
        within(d[r: r + 1], rows64(a[r: r + 1], sa[:, r: r + 1]), blocks64(b, sb), k)
    del d
    rows, cols = 300000, 7168
    x = torch.empty(rows, cols, dtype=BF, device="cuda")
    x[-200:] = torch.randn(200, cols, device="cuda").to(BF)
    x[:-200] = 1.0
    q, sf, qt, sft = nv.fp8_quantize(x, transpose=True)
    tail = rows - rows % 128 - 128
    q2, sf2, qt2, sft2 = nv.fp8_quantize(x[tail:].clone(), transpose=True)
    assert torch.equal(q[tail:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(sf[:, tail:], sf2)
    assert torch.equal(qt[:, tail:].view(torch.uint8), qt2.view(torch.uint8)) and torch.equal(sft[tail // 128:], sft2)
    q3, sf3 = nv.fp8_quantize(x)
    assert torch.equal(q3[tail:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(sf3, sf)
    nv.check_status()


def test_rows_of_more_than_2_gb(nv):
    """A weight gradient whose rows are longer than 2^31 bytes: a bulk copy's place in such a row would not fit its 32
    bits.  One expert of one row: D[0, c] = sum over r of a[0, r] b[c, r], ones and twos at known columns."""
    k = 2 ** 29 + 64
    if torch.cuda.mem_get_info()[0] < 90 * 2 ** 30:
        pytest.skip("needs 90 GB")
    one, two = 0x38, 0x40
    a = torch.full((1, 128), one, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    b = torch.zeros((k, 128), dtype=torch.uint8, device="cuda")
    at = torch.tensor([0, 1, 255, 256, 2 ** 28, 2 ** 29 - 1, 2 ** 29, 2 ** 29 + 1, k - 1], device="cuda")
    b[at, 5] = two
    b[at, 7] = one
    sfa, sfb = torch.ones((1, 1), device="cuda"), torch.ones((1, k), device="cuda")
    offsets = torch.tensor([0, 100], device="cuda")
    d = torch.full((1, 1, k), -1.0, device="cuda")
    nv.fp8_grouped_weight_grad(a, sfa, b.view(torch.float8_e4m3fn), sfb, offsets, d=d)
    nv.check_status()
    assert bool((d[0, 0, at] == 3.0).all())
    assert int((d != 0).sum()) == at.numel()


def test_misaligned_outputs_are_refused(nv):
    a, sa, b, sb = codes(1, 8, 128), scales(2, 1, 8), codes(3, 33, 128), scales(4, 1, 1)
    with pytest.raises(nv.NVFP4Error):
        nv.fp8_gemm(a, sa, b, sb, d=torch.empty(9, 33, dtype=BF, device="cuda")[1:])


@pytest.mark.parametrize("m,n,k", [(4, 512, 1024), (64, 512, 1024), (300, 520, 1024), (2000, 1536, 1024)])
def test_streams_at_once(nv, m, n, k):
    """Calls on four streams at a time give what each gives alone: there is no state between calls."""
    ops = [(codes(i, m, k), scales(i, 8, m), codes(10 + i, n, k), scales(20 + i, -(-n // 128), 8)) for i in range(4)]
    want = [nv.fp8_gemm(*o) for o in ops]
    streams = [torch.cuda.Stream() for _ in ops]
    torch.cuda.synchronize()
    got = [[] for _ in ops]
    for _ in range(6):
        for i, s in enumerate(streams):
            got[i].append(nv.fp8_gemm(*ops[i], stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for gs, w in zip(got, want) for g in gs)
    nv.check_status()


# ------------------------------------------------------------------ an expert layer
def layer(nv, x, ids, weights, w1, w2, dout, flags=0):
    """An expert layer with SiLU gates forward and backward: every step's operands and result by name."""
    r = {}
    experts, width, h = w1.shape
    inter = width // 2
    r["ro"], r["src"], r["pos"] = nv.moe_sort_by_expert(ids, experts, flags=flags)
    r["w1"], r["w2"] = nv.fp8_quantize_weight(w1, transpose=True, flags=flags), nv.fp8_quantize_weight(w2, transpose=True, flags=flags)
    r["xq"] = nv.fp8_quantize(x, src_rows=r["src"], row_offsets=r["ro"], transpose=True, flags=flags)
    r["gu"] = nv.fp8_grouped_gemm(*r["xq"][:2], r["ro"], *r["w1"][:2], flags=flags)
    g, u = r["gu"][:, :inter].float(), r["gu"][:, inter:].float()
    sg = torch.sigmoid(g)
    r["a"] = (g * sg * u).to(BF)
    r["aq"] = nv.fp8_quantize(r["a"], row_offsets=r["ro"], transpose=True)
    r["y"] = nv.fp8_grouped_gemm(*r["aq"][:2], r["ro"], *r["w2"][:2], flags=flags)
    r["out"] = nv.moe_combine(r["y"], r["pos"], weights, flags=flags)
    r["dy"], r["dweights"] = nv.moe_combine_backward(dout, r["y"], r["pos"], weights, flags=flags)
    r["dyq"] = nv.fp8_quantize(r["dy"], row_offsets=r["ro"], transpose=True, flags=flags)
    r["da"] = nv.fp8_grouped_gemm(*r["dyq"][:2], r["ro"], *r["w2"][2:], flags=flags)
    r["dw2"] = nv.fp8_grouped_weight_grad(*r["dyq"][2:], *r["aq"][2:], r["ro"], out_dtype=F32, flags=flags)
    da = r["da"].float()
    r["dgu"] = torch.cat((da * u * sg * (1 + g * (1 - sg)), da * g * sg), 1).to(BF)
    r["dguq"] = nv.fp8_quantize(r["dgu"], row_offsets=r["ro"], transpose=True)
    r["dxs"] = nv.fp8_grouped_gemm(*r["dguq"][:2], r["ro"], *r["w1"][2:], flags=flags)
    r["dw1"] = nv.fp8_grouped_weight_grad(*r["dguq"][2:], *r["xq"][2:], r["ro"], out_dtype=F32, flags=flags)
    r["dx"] = nv.moe_gather_backward(r["dxs"], r["pos"], flags=flags)
    return r


def inputs(seed, tokens, topk, experts, h, inter):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn(tokens, experts, generator=g, device="cuda") + torch.randn(1, experts, generator=g, device="cuda")
    p, ids = torch.topk(torch.softmax(logits, 1), topk, dim=1)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return (randn(tokens, h).to(BF), ids.to(torch.int32), p / p.sum(1, keepdim=True), randn(experts, 2 * inter, h) * 0.05, randn(experts, h, inter) * 0.05,
            (randn(tokens, h) * 1e-3).to(BF))


@pytest.mark.parametrize("tokens,topk,experts,h,inter", [(5, 2, 6, 128, 64), (300, 2, 7, 272, 144), (1200, 4, 16, 512, 256)])
def test_expert_layer_forward_and_backward(nv, tokens, topk, experts, h, inter):
    args = inputs(tokens, tokens, topk, experts, h, inter)
    x, ids, weights, w1, w2, dout = args
    r = layer(nv, *args)
    ro = r["ro"].tolist()
    src, pos = r["src"].long(), r["pos"].long()
    xq = ofp8.quantize_rows(x[src].float().cpu().numpy())
    assert np.array_equal(r["xq"][0].view(torch.uint8).cpu().numpy(), xq[0])
    at = 0
    for e in range(experts):
        lo, hi = ro[e], ro[e + 1]
        if hi == lo:
            assert bool((r["dw1"][e] == 0).all()) and bool((r["dw2"][e] == 0).all())
            continue
        cut = lambda q, s: rows64(q, s)[lo:hi]  # noqa: E731
        within(r["gu"][lo:hi], cut(*r["xq"][:2]), blocks64(r["w1"][0][e], r["w1"][1][e]), h)
        within(r["y"][lo:hi], cut(*r["aq"][:2]), blocks64(r["w2"][0][e], r["w2"][1][e]), inter)
        within(r["da"][lo:hi], cut(*r["dyq"][:2]), blocks64(r["w2"][0][e], r["w2"][1][e]).t(), h)
        within(r["dxs"][lo:hi], cut(*r["dguq"][:2]), blocks64(r["w1"][0][e], r["w1"][1][e]).t(), 2 * inter)
        n = hi - lo
        part = lambda q, s: rows64(q, s)[:, at: at + n]  # noqa: E731
        within(r["dw2"][e], part(*r["dyq"][2:]), part(*r["aq"][2:]), n)
        within(r["dw1"][e], part(*r["dguq"][2:]), part(*r["xq"][2:]), n)
        at += -(-n // 128) * 128
    y, dxs = r["y"].double(), r["dxs"].double()
    w = weights.double()
    dy = w.unsqueeze(2) * dout.double().unsqueeze(1)
    assert bool(((r["dy"].double()[pos] - dy).abs() <= dy.abs() * (2.0 ** -8 + 2.0 ** -23)).all())
    prod = dout.double().unsqueeze(1) * y[pos]
    assert bool(((r["dweights"].double() - prod.sum(2)).abs() <= (h + 8) * 2.0 ** -24 * prod.abs().sum(2)).all())
    dx = dxs[pos].sum(1)
    assert bool(((r["dx"].double() - dx).abs() <= dx.abs() * 2.0 ** -8 + topk * 2.0 ** -23 * dxs[pos].abs().sum(1)).all())
    nv.check_status()


def test_expert_layer_with_pdl_and_in_a_graph(nv):
    """The same chain with overlapping launches, and captured and replayed on new inputs: every result the same."""
    args, other = (list(inputs(s, 700, 2, 8, 256, 128)) for s in (1, 2))
    want, want2 = layer(nv, *args), layer(nv, *other)
    names = ("out", "dx", "dw1", "dw2", "dweights")
    got = layer(nv, *args, flags=nv.FLAG_PDL)
    assert all(torch.equal(got[k], want[k]) for k in names)
    held = [t.clone() for t in args]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layer(nv, *held, flags=nv.FLAG_PDL)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = layer(nv, *held, flags=nv.FLAG_PDL)
    for inp, ref in ((other, want2), (args, want), (other, want2)):
        for t, v in zip(held, inp):
            t.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], ref[k]) for k in names)
    nv.check_status()


def test_gradients_against_differences(nv):
    """On whole numbers up to 7 with a 7 in every block the codes are exact and so is every product: the gradients of
    loss = sum(y * c) equal its differences to the bit."""
    r = np.random.default_rng(3)

    def whole(*shape):
        v = r.integers(-6, 7, shape).astype(np.float32)
        v[..., ::16, :] = 7.0           # in every block of 128 along either axis
        v[..., :, ::16] = 7.0
        return torch.from_numpy(v).cuda()

    m, n, k = 160, 192, 256
    x, w, c = whole(m, k), whole(n, k), whole(m, n)

    def loss(x_, w_):
        y = nv.fp8_gemm(*nv.fp8_quantize(x_), *nv.fp8_quantize_weight(w_), out_dtype=F32)
        assert torch.equal(y.double(), x_.double() @ w_.double().t())
        return float((y.double() * c.double()).sum())

    wt = nv.fp8_quantize_weight(w, transpose=True)[2:]
    cq = nv.fp8_quantize(c, transpose=True)
    xt = nv.fp8_quantize(x, rows=False, transpose=True)
    dx = nv.fp8_gemm(*cq[:2], *wt, out_dtype=F32)
    dw = nv.fp8_gemm(*cq[2:], *xt, block_b=1, out_dtype=F32)
    base = loss(x, w)
    for _ in range(12):
        i, j, t = int(r.integers(n)), int(r.integers(k)), int(r.integers(m))
        if abs(float(w[i, j])) < 6 and abs(float(x[t, j])) < 6:
            w2, x2 = w.clone(), x.clone()
            w2[i, j] += 1
            x2[t, j] += 1
            assert loss(x, w2) - base == float(dw[i, j]) and loss(x2, w) - base == float(dx[t, j])
    total = torch.zeros_like(dw)
    for _ in range(2):
        nv.fp8_gemm(*cq[2:], *xt, block_b=1, d=total, accumulate=True)
    assert torch.equal(total, 2 * dw)
    off = torch.tensor([0, 70, 70, m], device="cuda")
    ct, xt = (nv.fp8_quantize(v, row_offsets=off, rows=False, transpose=True) for v in (c, x))
    per = nv.fp8_grouped_weight_grad(*ct, *xt, off, out_dtype=F32)
    assert torch.equal(per.double(), torch.stack([c[a:b].double().t() @ x[a:b].double() for a, b in ((0, 70), (70, 70), (70, m))]))
    again = per.clone()
    nv.fp8_grouped_weight_grad(*ct, *xt, off, d=again, accumulate=True)
    assert torch.equal(again, 2 * per)
    nv.check_status()
