"""The draw of a token per row on the GPU against the fp64 form of oracle/block.py.

Bounds, fixed by the arithmetic.  x = (z - m) log2(e) / T carries three roundings of 2^-24 each and lies in
[-32, 0], so 2^x is off by at most 32 * 3 * 2^-24 * ln 2 < 2^-17.9 of itself, the hardware's 2^x by 2^-22 and
the whole number by 2^-31 of the largest weight: every sum of weights is within REL = 2^-17 of its fp64
value (plus vocab * 2^-31 of the largest weight, below 2^-17 of a sum for these rows).  A token drawn at u
must therefore cover u in the fp64 distribution up to 2 REL on either side, taken over the kept set of
filters that are REL stricter or looser; a token on the edge of top-p moves the whole distribution by
less than 2 REL more.  DELTA = 2^-14 covers the sum.  Where logits are whole multiples of the
temperature's step the token is known exactly."""
import numpy as np
import pytest
import torch

from oracle import block

pytestmark = pytest.mark.gpu

DELTA = 2.0 ** -14
STEP = float(np.float32(1.4426950408889634))     # this temperature makes x = z - m


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_bf16_gb300 as m
    return m


def vec(v, rows, dtype=torch.float32):
    if v is None:
        return None
    a = np.broadcast_to(np.asarray(v), (rows,))
    return torch.tensor(a.tolist(), dtype=dtype, device="cuda")


def draw(nv, z, u, t=None, k=None, p=None, mp=None, **kw):
    rows = z.shape[0]
    tok, lp = nv.sample_tokens(z, vec(u, rows), vec(t, rows), vec(k, rows, torch.int32), vec(p, rows), vec(mp, rows), **kw)
    return tok.cpu().numpy(), lp.cpu().numpy()


def covers(z, u, tok, lp, t=1.0, k=0, p=1.0, mp=0.0):
    """tok may be drawn at u from the row z (see above), and lp is its log-probability."""
    loose, _ = block.kept(z, t, k, p + DELTA if p < 1 else 1.0, mp * (1 - DELTA))
    tight, _ = block.kept(z, t, k, p - DELTA if p < 1 else 1.0, mp * (1 + DELTA))
    assert loose[tok] > 0, "a filtered token"
    ok = []
    for w in (loose, tight):
        c = np.cumsum(w) / w.sum()
        # (the edge token of a filter may be missing from the tight set: then it covers nothing there)
        ok.append((c[tok - 1] if tok else 0.0) - DELTA <= u <= c[tok] + DELTA)
    assert any(ok), (u, tok)
    probs = [np.log(loose[tok] / w.sum()) for w in (loose, tight)]
    assert min(probs) - DELTA <= lp <= max(probs) + DELTA
    return True


def logits(rows, v, dtype, spread, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, v + pad, generator=g) * spread
    z[:, : min(4, v)] += 2 * spread
    return z.to(dtype).cuda()[:, pad // 2: pad // 2 + v]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,v,pad", [(1, 1, 0), (1, 2, 1), (3, 7, 0), (2, 33, 5), (5, 1000, 3), (1, 4095, 0), (9, 8200, 6),
                                        (2, 32000, 0), (1, 50001, 9), (40, 20011, 1), (170, 9000, 0), (400, 4100, 2)])
@pytest.mark.parametrize("name", ["none", "top_k", "top_p", "min_p", "all"])
def test_draw(nv, dtype, rows, v, pad, name):
    rng = np.random.default_rng(rows + v)
    z = logits(rows, v, dtype, 2.0, rows * 7 + v, pad)
    u = rng.random(rows).astype(np.float32)
    t = (0.5 + rng.random(rows)).astype(np.float32)
    k = rng.integers(1, 80, rows).astype(np.int32) if name in ("top_k", "all") else None
    p = (0.5 + 0.5 * rng.random(rows)).astype(np.float32) if name in ("top_p", "all") else None
    mp = (0.2 * rng.random(rows)).astype(np.float32) if name in ("min_p", "all") else None
    tok, lp = draw(nv, z, u, t, k, p, mp)
    zz = z.double().cpu().numpy()
    for r in range(min(rows, 40)):
        assert 0 <= tok[r] < v
        covers(zz[r], float(u[r]), int(tok[r]), float(lp[r]), float(t[r]), 0 if k is None else int(k[r]),
               1.0 if p is None else float(p[r]), 0.0 if mp is None else float(mp[r]))


@pytest.mark.parametrize("v", [131072, 200003])
def test_a_long_flat_row(nv, v):
    """top-p keeps tens of thousands of tokens, and classes hold more keys than are sorted at once."""
    z = logits(2, v, torch.bfloat16, 0.3, 5)
    u = np.array([0.3, 0.9], dtype=np.float32)
    tok, lp = draw(nv, z, u, None, None, 0.9, None)
    for r in range(2):
        covers(z[r].double().cpu().numpy(), float(u[r]), int(tok[r]), float(lp[r]), p=float(np.float32(0.9)))


@pytest.mark.parametrize("rows", [1, 40, 90, 170, 400])
def test_a_row_does_not_depend_on_its_batch(nv, rows):
    """The same row alone and in batches that give it 1, 2, 4 or 8 CTAs: the same token, bit for bit the
    same log-probability."""
    z = logits(rows, 40003, torch.float32, 2.0, 11)
    rng = np.random.default_rng(0)
    u = rng.random(rows).astype(np.float32)
    kw = dict(t=np.float32(0.8), k=50, p=np.float32(0.9), mp=np.float32(0.01))
    for f in (kw, dict(t=np.float32(1.2)), dict(p=np.float32(0.95))):
        tok, lp = draw(nv, z, u, **f)
        for r in range(0, rows, 23):
            a, b = draw(nv, z[r:r + 1], u[r:r + 1], **f)
            assert a[0] == tok[r] and b[0] == lp[r]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [6, 5000, 131072])
def test_equal_logits_are_cut_by_index(nv, v, dtype):
    """Every token ties: top-k keeps the first k, top-p the first ceil(p v), and the draw is floor(u n)."""
    z = torch.full((4, v), 3.25, dtype=dtype, device="cuda")
    u = np.array([0.0, 0.3, 0.61, 0.999], dtype=np.float32)
    for k in (1, 5):
        tok, lp = draw(nv, z, u, k=k)
        assert tok.tolist() == [int(x * k) for x in u.astype(float)]
        assert np.allclose(lp, -np.log(k), atol=1e-6)
    n = -(-v // 2)
    tok, lp = draw(nv, z, u, p=0.5)
    assert tok.tolist() == [int(x * n) for x in u.astype(float)]
    tok, _ = draw(nv, z, u)
    assert tok.tolist() == [int(x * v) for x in u.astype(float)]
    tok, _ = draw(nv, z, u, k=v, p=1.0, mp=1.0)
    assert tok.tolist() == [int(x * v) for x in u.astype(float)]


def test_ties_at_the_cut_across_a_split_class(nv):
    """16 values less than 1/32 apart, thousands of tokens each, interleaved: the class must be split and
    the ties at the cut taken by index.  Weights are within 1.6 % of each other, so the fp64 form gives
    the kept set exactly and the draw is checked inside it."""
    v = 120000
    idx = torch.arange(v)
    z = (5.0 - (idx * 7 % 16).float() * 2.0 ** -10).unsqueeze(0).repeat(3, 1).cuda()
    zz = z[0].double().cpu().numpy()
    u = np.array([0.05, 0.5, 0.98], dtype=np.float32)
    for k, p in ((30000, None), (7500, None), (60001, 0.5), (None, 0.25)):
        tok, lp = draw(nv, z, u, k=k, p=p)
        w, _ = block.kept(zz, 1.0, k or 0, 1.0 if p is None else p, 0.0)
        c = np.cumsum(w) / w.sum()
        for r in range(3):
            assert w[tok[r]] > 0
            assert (c[tok[r]] - w[tok[r]] / w.sum()) - 1e-5 <= u[r] <= c[tok[r]] + 1e-5


def test_weights_that_are_powers_of_two(nv):
    """x = -0, -1, -2, ... exactly: the draw is known for any u away from the edges."""
    z = torch.tensor([[-3.0, -1.0, 0.0, -2.0, -1.0, -40.0, float("-inf")]], device="cuda")
    w = np.array([1 / 8, 1 / 2, 1, 1 / 4, 1 / 2, 0, 0])

    def expect(keep, u):
        c = np.cumsum(w * keep)
        return int(np.searchsorted(c, u * c[-1], side="right"))

    for u in (0.0, 0.03, 0.2, 0.33, 0.5, 0.8, 0.93, 0.999):
        for kw, keep in ((dict(), [1, 1, 1, 1, 1, 1, 0]), (dict(k=2), [0, 1, 1, 0, 0, 0, 0]), (dict(k=3), [0, 1, 1, 0, 1, 0, 0]),
                         (dict(p=0.7), [0, 1, 1, 0, 1, 0, 0]), (dict(p=0.5), [0, 1, 1, 0, 0, 0, 0]),
                         (dict(k=3, p=0.7), [0, 1, 1, 0, 0, 0, 0]), (dict(mp=0.4), [0, 1, 1, 0, 1, 0, 0]),
                         (dict(mp=0.2, p=0.99), [0, 1, 1, 1, 1, 0, 0]), (dict(p=0.0), [0, 0, 1, 0, 0, 0, 0]),
                         (dict(mp=2.0), [0, 0, 1, 0, 0, 0, 0]), (dict(k=1), [0, 0, 1, 0, 0, 0, 0])):
            tok, lp = draw(nv, z, u, t=STEP, **kw)
            want = expect(np.array(keep), u)
            assert tok[0] == want, (u, kw, tok[0], want)
            assert abs(lp[0] - np.log(w[want] / (w * keep).sum())) < 1e-5


def test_greedy_and_extreme_temperatures(nv):
    z = torch.tensor([[1.0, 7.0, 3.0, 7.0], [2.0, -5.0, 2.0, 1.9]], device="cuda")
    for t in (0.0, -1.0, float("nan"), 1e-30, 1e-42):
        tok, lp = draw(nv, z, [0.0, 0.0], t=t)
        assert tok.tolist() == [1, 0]
    tok, lp = draw(nv, z, [0.9, 0.9], t=0.0)
    assert tok.tolist() == [1, 0] and not lp.any()
    tok, _ = draw(nv, z, [0.9, 0.9], t=1e-30)                     # two largest logits share the weight
    assert tok.tolist() == [3, 2]
    for t in (1e30, float("inf")):                                # every token as likely as any other
        tok, _ = draw(nv, z, [0.3, 0.8], t=t)
        assert tok.tolist() == [1, 3]


def test_infinities_nan_and_empty_rows(nv):
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[nan, -inf, nan, -inf, -inf], [nan, 1.0, -inf, nan, -inf], [2.0, inf, nan, inf, 1e38],
                      [-inf, -inf, -3e38, -inf, nan], [3e38, -3e38, 3e38, 0.0, nan]], device="cuda")
    for kw in (dict(), dict(k=3), dict(p=0.9), dict(k=4, p=0.9, mp=0.1), dict(t=0.0), dict(t=inf)):
        lo, lpl = draw(nv, z, 0.0, **kw)
        hi, lph = draw(nv, z, 0.75, **kw)
        assert lo[0] == hi[0] == -1 and lpl[0] == lph[0] == -inf
        assert lo[1] == hi[1] == 1 and lpl[1] == 0.0
        assert lo[2] == 1 and hi[2] == (1 if kw.get("t") == 0.0 else 3)
        assert lo[3] == hi[3] == 2
    tok, _ = draw(nv, z[4:], 0.75)
    assert tok[0] == 2
    for dtype in (torch.float32, torch.bfloat16):
        long = torch.full((2, 60000), -inf, dtype=dtype, device="cuda")
        long[1, 59999] = -2.0
        tok, _ = draw(nv, long, 0.5, k=20, p=0.9)
        assert tok.tolist() == [-1, 59999]
    tok, lp = nv.sample_tokens(torch.empty(0, 50, device="cuda"), torch.empty(0, device="cuda"))
    assert tok.shape == lp.shape == (0,)


def test_random_numbers_outside_their_range(nv):
    z = torch.tensor([[0.0, 1.0, 0.5]], device="cuda")
    assert draw(nv, z, [-0.5])[0][0] == 0 and draw(nv, z, [1.0])[0][0] == 2 and draw(nv, z, [7.0])[0][0] == 2
    assert draw(nv, z, [float("nan")])[0][0] == 0
    assert draw(nv, z, [1.0], k=2)[0][0] == 2 and draw(nv, z, [1.0], k=1)[0][0] == 1


def test_the_draw_follows_the_distribution(nv):
    """2^14 draws at evenly spaced numbers: each token's share is its probability to one draw."""
    n, v = 1 << 14, 300
    row = logits(1, v, torch.float32, 1.5, 2)
    u = (np.arange(n) + 0.5) / n
    tok, _ = draw(nv, row.expand(n, v), u.astype(np.float32), t=0.9, k=40, p=0.95)
    w, _ = block.kept(row[0].double().cpu().numpy(), float(np.float32(0.9)), 40, float(np.float32(0.95)))
    got = np.bincount(tok, minlength=v)
    assert np.all(np.abs(got - n * w / w.sum()) <= 2 + n * DELTA)


def test_another_stream_and_pdl(nv):
    z = logits(8, 30000, torch.bfloat16, 2.0, 9)
    u = vec(np.linspace(0, 0.99, 8), 8)
    want, _ = nv.sample_tokens(z, u, top_p=vec(0.9, 8))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    tok = torch.empty_like(want)
    lp = torch.empty(8, device="cuda")
    top_p = vec(0.9, 8)
    torch.cuda.synchronize()
    nv.sample_tokens(z, u, top_p=top_p, tokens=tok, logprobs=lp, stream=s, flags=nv.FLAG_PDL)
    s.synchronize()
    assert torch.equal(tok, want)


def test_offsets_past_32_bits(nv):
    """Rows 2^30 + 3 elements apart: the last one begins past 2^31."""
    z = logits(3, 20000, torch.bfloat16, 2.0, 21)
    ld = (1 << 30) + 3
    far = torch.empty(2 * ld + 20000, dtype=torch.bfloat16, device="cuda").as_strided((3, 20000), (ld, 1))
    far.copy_(z)
    for kw in (dict(), dict(k=50), dict(p=0.9, mp=0.01)):
        a, b = draw(nv, z, [0.2, 0.5, 0.8], **kw), draw(nv, far, [0.2, 0.5, 0.8], **kw)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_fallback_rows_beside_ordinary_ones(nv):
    """A batch that mixes rows whose cut is found in the bracket with rows that need the whole row's classes
    (equal logits, a k near the end), so that CTAs of different rows take different ways at once."""
    v, rows = 30000, 60
    z = logits(rows, v, torch.float32, 2.0, 33)
    z[::3] = 1.5
    k = np.where(np.arange(rows) % 5 == 0, v - 3, 40).astype(np.int32)
    u = np.linspace(0.01, 0.97, rows).astype(np.float32)
    p = np.full(rows, 0.8, dtype=np.float32)
    tok, lp = draw(nv, z, u, k=k, p=p)
    zz = z.double().cpu().numpy()
    for r in range(rows):
        if r % 3 == 0:       # ceil(0.8 k) equal tokens (k may be v - 3), by index
            n = int(np.ceil(np.float64(p[r]) * int(k[r]) - 1e-9))
            assert tok[r] == int(float(u[r]) * n), r
        else:
            covers(zz[r], float(u[r]), int(tok[r]), float(lp[r]), k=int(k[r]), p=float(p[r]))
