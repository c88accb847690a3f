"""Pins for oracle/block.py: the norms and the gated product against torch's autograd in fp64 and central
differences, the interleaved layout against hand-worked rows, the draw against hand-worked rows and exact
rationals."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import block


def _norm_case(seed=0, m=4, n=12, gate="token"):
    rng = np.random.default_rng(seed)
    d = dict(x=rng.standard_normal((m, n)), y=rng.standard_normal((m, n)), w_post=rng.standard_normal(n),
             w_pre=rng.standard_normal(n), gate=rng.standard_normal((m, n) if gate == "token" else n))
    return d, rng.standard_normal((m, n)), rng.standard_normal((m, n))


def test_norm_of_a_hand_worked_row():
    r, h = block.block_norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), eps=0.0)
    rms = np.sqrt(12.5)
    assert np.allclose(h, [[3 / rms, 8 / rms]]) and np.array_equal(r, [[3.0, 4.0]])
    # the branch alone: y normalised, scaled by 0.5, gated by 2 and 4, added
    r, h = block.block_norm(np.zeros((1, 2)), None, np.array([[3.0, 4.0]]), np.zeros(2), np.array([2.0, 4.0]), 0.5, 0.0, 1.0)
    assert h is None and np.allclose(r, [[3 / rms, 8 / rms]])


@pytest.mark.parametrize("gate", ["token", "channel"])
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_norm_gradients_against_autograd_and_differences(gate, offset):
    d, dh, dr = _norm_case(1, gate=gate)
    scale, eps = 0.6, 1e-3
    t = {k: torch.from_numpy(v).requires_grad_() for k, v in d.items()}

    def rms(v, w):
        return v * torch.rsqrt((v * v).mean(1, keepdim=True) + eps) * (offset + w)

    r = t["x"] + scale * rms(t["y"], t["w_post"]) * t["gate"]
    ((rms(r, t["w_pre"]) * torch.from_numpy(dh)).sum() + (r * torch.from_numpy(dr)).sum()).backward()
    got = block.block_norm_backward(dh, dr, r.detach().numpy(), d["w_pre"], d["y"], d["w_post"], d["gate"], scale, eps, offset)
    for name, g in zip(("x", "y", "w_pre", "w_post", "gate"), got):
        assert np.allclose(g, t[name].grad.numpy(), rtol=1e-10, atol=1e-12), name

    def loss(a):
        rr, hh = block.block_norm(a["x"], a["w_pre"], a["y"], a["w_post"], a["gate"], scale, eps, offset)
        return np.sum(rr * dr) + np.sum(hh * dh)

    rng = np.random.default_rng(9)
    for name, g in zip(("x", "y", "w_pre", "w_post", "gate"), got):
        v = rng.standard_normal(d[name].shape)
        num = (loss({**d, name: d[name] + 1e-6 * v}) - loss({**d, name: d[name] - 1e-6 * v})) / 2e-6
        assert abs(num - np.sum(g * v)) <= 1e-7 * (1 + abs(num)), name


def test_norm_gradients_of_absent_parts():
    d, dh, dr = _norm_case(2)
    dx, dy, dw, dp, dg = block.block_norm_backward(None, dr, d["x"], None, d["y"], None, None, 2.0)
    assert np.array_equal(dx, dr) and np.array_equal(dy, 2.0 * dr) and dw is dp is dg is None
    dx, dy, dw, dp, dg = block.block_norm_backward(dh, None, d["x"], d["w_pre"])
    assert dy is dp is dg is None and np.allclose(np.sum(dx * d["x"], axis=1), 0.0, atol=1e-5)  # h keeps its length


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_activations_against_torch(kind):
    g = torch.linspace(-12, 12, 2001, dtype=torch.float64, requires_grad=True)
    f = torch.nn.functional.silu(g) if kind == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
    f.sum().backward()
    a, da = block.activation(g.detach().numpy(), kind)
    assert np.allclose(a, f.detach().numpy(), atol=1e-13) and np.allclose(da, g.grad.numpy(), atol=1e-12)
    # what the tolerances of the GPU tests take for granted
    assert np.abs(da).max() <= 1.13
    assert np.abs(np.diff(da) / np.diff(g.detach().numpy())).max() <= 1.0


def test_gate_and_up_rows_alternate_in_groups_of_sixteen():
    c = np.arange(64)[None, :]
    g, u = block.split_gate_up(c)
    assert g.tolist() == [list(range(0, 16)) + list(range(32, 48))]
    assert u.tolist() == [list(range(16, 32)) + list(range(48, 64))]
    assert np.array_equal(block.join_gate_up(g, u), c)


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gated_product_and_gradients_against_autograd(kind):
    rng = np.random.default_rng(3)
    a, b = rng.standard_normal((3, 8)), rng.standard_normal((64, 8))
    dh = rng.standard_normal((3, 32))
    alpha = (0.7, 1.3)
    c = torch.from_numpy(a @ b.T).requires_grad_()
    v = c.view(3, 2, 2, 16)
    g, u = alpha[0] * v[:, :, 0].reshape(3, 32), alpha[1] * v[:, :, 1].reshape(3, 32)
    f = torch.nn.functional.silu(g) if kind == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
    h = f * u
    h.backward(torch.from_numpy(dh))
    assert np.allclose(block.gated(a, b, alpha, kind), h.detach().numpy())
    dgu, h2 = block.gated_backward(a, b, alpha, dh, kind)
    # dgu is the gradient of the products themselves, alpha applied: d/dc = alpha * dgu
    factor = block.join_gate_up(np.full((3, 32), alpha[0]), np.full((3, 32), alpha[1]))
    assert np.allclose(dgu * factor, c.grad.numpy()) and np.allclose(h2, h.detach().numpy())


def test_draw_of_hand_worked_rows():
    ln2 = np.log(2.0)
    z = np.array([-3.0, -1.0, 0.0, -2.0, -1.0]) * ln2             # weights 1/8 1/2 1 1/4 1/2
    w, order = block.kept(z)
    assert order.tolist() == [2, 1, 4, 3, 0] and np.allclose(w, [1 / 8, 1 / 2, 1, 1 / 4, 1 / 2])
    assert np.nonzero(block.kept(z, top_k=2)[0])[0].tolist() == [1, 2]              # the tie goes to index 1
    assert np.nonzero(block.kept(z, top_p=0.5)[0])[0].tolist() == [1, 2]            # 1 < 1.1875 <= 1.5
    assert np.nonzero(block.kept(z, top_p=0.7)[0])[0].tolist() == [1, 2, 4]
    assert np.nonzero(block.kept(z, top_k=3, top_p=0.7)[0])[0].tolist() == [1, 2]   # of the three: 1.4 of 2
    assert np.nonzero(block.kept(z, min_p=0.3)[0])[0].tolist() == [1, 2, 4]
    assert np.nonzero(block.kept(z, top_p=0.0)[0])[0].tolist() == [2]
    assert np.nonzero(block.kept(z, min_p=5.0)[0])[0].tolist() == [2]
    assert np.nonzero(block.kept(z, temperature=0.0)[0])[0].tolist() == [2]
    assert np.allclose(block.kept(z, temperature=2.0)[0], np.sqrt([1 / 8, 1 / 2, 1, 1 / 4, 1 / 2]))
    total = Fraction(19, 8)
    edges = [Fraction(1, 8), Fraction(5, 8), Fraction(13, 8), Fraction(15, 8), total]
    for u in np.linspace(0.01, 0.99, 37):
        want = next(i for i, e in enumerate(edges) if Fraction(float(u)) * total < e)
        assert block.draw(w, u) == want


def test_draw_of_rows_with_infinities_and_nothing():
    inf, nan = np.inf, np.nan
    assert block.draw(block.kept(np.array([-inf, nan]))[0], 0.5) == -1
    w, _ = block.kept(np.array([1.0, inf, nan, inf]))
    assert w.tolist() == [0.0, 1.0, 0.0, 1.0]
    assert block.draw(w, 0.4) == 1 and block.draw(w, 0.6) == 3
    w, _ = block.kept(np.array([nan, 2.0, -inf]))
    assert w.tolist() == [0.0, 1.0, 0.0] and block.draw(w, 0.99) == 1
    assert block.draw(np.zeros(0), 0.5) == -1
