"""Pins for oracle/fp8.py: hand-worked blocks, torch's e4m3 cast, layouts, the bounds that its docstring and the
header state, the MoE gradients against autograd and differences."""
import numpy as np
import torch

from oracle import fp8
from oracle.formats import e4m3_decode

F32 = np.float32


def test_encode_against_torch_and_every_code():
    c = np.arange(256, dtype=np.uint8)
    v = e4m3_decode(c)
    ok = np.isfinite(v)
    assert np.array_equal(fp8.encode(v[ok].astype(F32)), c[ok])
    assert fp8.encode(F32(np.nan)) == 0x7F and fp8.encode(F32(1e9)) == 0x7E and fp8.encode(F32(-1e9)) == 0xFE
    x = (np.random.default_rng(0).standard_normal(20000) * np.exp2(np.random.default_rng(1).integers(-12, 9, 20000))).astype(F32)
    x = x[np.abs(x) <= 448]
    assert np.array_equal(fp8.encode(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_hand_worked_block():
    x = np.zeros((2, 130), F32)
    x[0, 0], x[0, 1], x[0, 2] = 896.0, -2.0, 3.0     # scale 2: codes of 448, -1, 1.5
    x[1, 129] = 7.0                                   # the short last block: scale 1/64
    q, s = fp8.quantize_rows(x)
    assert s.shape == (2, 2) and s[0, 0] == 2.0 and s[1, 1] == F32(7.0) / F32(448.0) == F32(1 / 64)
    assert list(e4m3_decode(q[0, :4])) == [448.0, -1.0, 1.5, 0.0] and e4m3_decode(q[1, 129]) == 448.0
    assert s[0, 1] == s[1, 0] == F32(2.0 ** -100) / F32(448.0)      # blocks of zeros
    assert np.array_equal(fp8.rows_value(q, s), x)


def test_columns_are_the_rows_of_the_transpose():
    x = np.random.default_rng(2).standard_normal((256, 50)).astype(F32)
    q, s = fp8.quantize_columns(x)
    qr, sr = fp8.quantize_rows(np.ascontiguousarray(x.T))
    assert np.array_equal(q, qr) and np.array_equal(s, sr)


def test_experts_begin_at_multiples_of_128():
    x = np.random.default_rng(3).standard_normal((133, 16)).astype(F32)
    ro = np.array([0, 3, 3, 132])
    q, s = fp8.quantize_columns(x, ro)
    assert q.shape == (16, 256 + 3 * 128) and s.shape == (5, 16)
    for lo, hi, at in ((0, 3, 0), (3, 131, 128), (131, 132, 256)):
        qe, se = fp8.quantize_columns(x[lo:hi])
        assert np.array_equal(q[:, at: at + 128], qe) and np.array_equal(s[at // 128: at // 128 + 1], se)
    assert (q[:, 384:] == 0).all()


def test_blocks_and_their_transpose():
    w = np.random.default_rng(4).standard_normal((200, 300)).astype(F32)
    q, s = fp8.quantize_blocks(w)
    qt, st = fp8.quantize_blocks(np.ascontiguousarray(w.T))
    assert s.shape == (2, 3) and np.array_equal(q.T, qt) and np.array_equal(s.T, st)
    for i in range(2):
        for j in range(3):
            assert s[i, j] == F32(np.abs(w[128 * i: 128 * (i + 1), 128 * j: 128 * (j + 1)]).max()) / F32(448.0)


def test_value_is_within_half_a_step():
    """|value - x| <= |x| 2^-4 above the normal range's foot, amax / 448 * 2^-10 below, and the three roundings of
    2^-24 before the code's."""
    x = (np.random.default_rng(5).standard_normal((64, 256)) * np.exp2(np.random.default_rng(6).integers(-20, 3, (64, 256)))).astype(F32)
    q, s = fp8.quantize_rows(x)
    v = fp8.rows_value(q, s)
    amax = np.repeat(np.abs(x).reshape(64, 2, 128).max(2), 128, axis=1).astype(np.float64)
    x = x.astype(np.float64)
    tol = np.maximum(np.abs(x) * 2.0 ** -4, amax / 448 * 2.0 ** -10) + np.abs(x) * 3 * 2.0 ** -24
    assert (np.abs(v - x) <= tol).all()


def test_non_finite_blocks_give_nothing_finite():
    x = np.ones((3, 256), F32)
    x[0, 3], x[1, 200], x[2, 0] = np.inf, np.nan, -np.inf
    with np.errstate(invalid="ignore"):
        v = fp8.rows_value(*fp8.quantize_rows(x))
    finite = np.isfinite(v)
    assert not finite[0, :128].any() and not finite[1, 128:].any() and not finite[2, :128].any()
    assert finite[0, 128:].all() and finite[1, :128].all()


def test_moe_gradients_against_autograd_and_differences():
    r = np.random.default_rng(7)
    pos = np.array([[2, 0], [-1, 4], [3, 1]])
    x, y, w, dout, dxs = (r.standard_normal(s) for s in ((3, 5), (6, 5), (3, 2), (3, 5), (6, 5)))
    ty, tw, tx = (torch.from_numpy(v).requires_grad_() for v in (y, w, x))
    out = torch.stack([sum(tw[t, j] * ty[pos[t, j]] for j in range(2) if pos[t, j] >= 0) for t in range(3)])
    (out * torch.from_numpy(dout)).sum().backward()
    dy, dw = fp8.combine_grad(dout, y, pos, w)
    assert np.allclose(dy, ty.grad.numpy()) and np.allclose(dw, tw.grad.numpy())
    loss = sum((tx[t] * torch.from_numpy(dxs[pos[t, j]])).sum() for t in range(3) for j in range(2) if pos[t, j] >= 0)
    loss.backward()
    assert np.allclose(fp8.gather_grad(dxs, pos), tx.grad.numpy())

    def combined(y_, w_):
        return sum((w_[t, j] * y_[pos[t, j]] * dout[t]).sum() for t in range(3) for j in range(2) if pos[t, j] >= 0)

    for arr, grad, f in ((y, dy, lambda v: combined(v, w)), (w, dw, lambda v: combined(y, v))):
        for i in np.ndindex(arr.shape):
            step = np.zeros_like(arr)
            step[i] = 1e-3
            assert abs((f(arr + step) - f(arr - step)) / 2e-3 - grad[i]) < 1e-9


def test_product_slack_covers_fp32_sums():
    r = np.random.default_rng(8)
    a, b = (e4m3_decode(c).astype(F32) for c in (r.integers(0, 0x7F, (8, 1024)), r.integers(0, 0x7F, (9, 1024))))
    got = np.zeros((8, 9), F32)
    for k0 in range(0, 1024, 128):
        part = np.zeros((8, 9), F32)
        for k in range(k0, k0 + 128):
            part = (part + np.outer(a[:, k], b[:, k])).astype(F32)
        got = (got + part).astype(F32)
    want = a.astype(np.float64) @ b.astype(np.float64).T
    assert (np.abs(got - want) <= fp8.product_slack(1024) * want).all()
