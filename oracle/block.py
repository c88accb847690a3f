"""Plain numpy fp64 forms of the operators around a decoder block's products: the norms before and
after a block with its gate and residual sum, the gated product of a feed-forward block, and the draw
of a token from its logits.  Each takes and returns plain arrays (a value per element, any layout that
the CUDA path packs is unpacked by the caller) and follows the formulas stated at the entry points in
include/nvfp4.h.  Pinned by tests/test_oracle_block.py."""
from __future__ import annotations

import numpy as np

F64 = np.float64


# ------------------------------------------------------------------ norms
def _rms(v, eps):
    """v / sqrt(mean(v^2) + eps), and the reciprocal root itself."""
    rstd = 1.0 / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)
    return v * rstd, rstd


def block_norm(x, w_pre=None, y=None, w_post=None, gate=None, scale=1.0, eps=1e-6, offset=0.0):
    """(r, h) of one pass; h is None without w_pre."""
    r = np.asarray(x, F64)
    if y is not None:
        p = np.asarray(y, F64)
        if w_post is not None:
            p = _rms(p, eps)[0] * (offset + np.asarray(w_post, F64))
        if gate is not None:
            p = p * np.asarray(gate, F64)
        r = r + scale * p
    h = None if w_pre is None else _rms(r, eps)[0] * (offset + np.asarray(w_pre, F64))
    return r, h


def block_norm_backward(dh, dr, r, w_pre=None, y=None, w_post=None, gate=None, scale=1.0, eps=1e-6, offset=0.0):
    """(dx, dy, dw_pre, dw_post, dgate) from the stored stream r."""
    r = np.asarray(r, F64)
    g = np.zeros_like(r) if dr is None else np.asarray(dr, F64).copy()
    dw_pre = dw_post = dgate = dy = None
    if dh is not None:
        d = np.asarray(dh, F64)
        xn, rstd = _rms(r, eps)
        dw_pre = np.sum(d * xn, axis=0)
        d = d * (offset + np.asarray(w_pre, F64))
        g += rstd * (d - xn * np.mean(d * xn, axis=1, keepdims=True))
    if y is not None:
        y = np.asarray(y, F64)
        yn, rstd = _rms(y, eps) if w_post is not None else (y, 1.0)
        w = offset + np.asarray(w_post, F64) if w_post is not None else 1.0
        b = scale * g
        if gate is not None:
            gate = np.asarray(gate, F64)
            dgate = b * yn * w
            if gate.ndim == 1:
                dgate = dgate.sum(axis=0)
            b = b * gate
        dy = b
        if w_post is not None:
            dw_post = np.sum(b * yn, axis=0)
            e = b * w
            dy = rstd * (e - yn * np.mean(e * yn, axis=1, keepdims=True))
    return g, dy, dw_pre, dw_post, dgate


# ------------------------------------------------------------------ gated product
def activation(g, kind):
    """(f, f') of the activation at g."""
    g = np.asarray(g, F64)
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if kind == "gelu_tanh":
        k = np.sqrt(2.0 / np.pi)
        th = np.tanh(k * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th ** 2) * k * (1.0 + 3 * 0.044715 * g ** 2)
    raise ValueError(kind)


def split_gate_up(c):
    """The gate and the up columns of a product with an interleaved weight (groups of 16)."""
    v = c.reshape(c.shape[0], -1, 2, 16)
    return v[:, :, 0].reshape(c.shape[0], -1), v[:, :, 1].reshape(c.shape[0], -1)


def join_gate_up(g, u):
    """Inverse of split_gate_up."""
    m = g.shape[0]
    return np.stack((g.reshape(m, -1, 16), u.reshape(m, -1, 16)), axis=2).reshape(m, -1)


def gated(a, b, alpha, kind):
    """h = act(alpha0 a Bg^T) * (alpha1 a Bu^T) for a dequantised a [m, k] and interleaved b [2i, k]."""
    g, u = split_gate_up(np.asarray(a, F64) @ np.asarray(b, F64).T)
    return activation(F64(alpha[0]) * g, kind)[0] * (F64(alpha[1]) * u)


def gated_backward(a, b, alpha, dh, kind):
    """(gradients of the two pre-activations, interleaved [m, 2i]; h)."""
    g, u = split_gate_up(np.asarray(a, F64) @ np.asarray(b, F64).T)
    g, u = F64(alpha[0]) * g, F64(alpha[1]) * u
    f, df = activation(g, kind)
    dh = np.asarray(dh, F64)
    return join_gate_up(dh * u * df, dh * f), f * u


# ------------------------------------------------------------------ draw of a token
def kept(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The distribution one row's token is drawn from: (weights relative to the largest, 0 where a
    filter or a NaN removes the token; the order of the tokens, likeliest first, ties by index)."""
    z = np.asarray(logits, F64).copy()
    z[np.isnan(z)] = -np.inf
    m = z.max() if z.size else -np.inf
    if m == -np.inf:
        return np.zeros_like(z), np.arange(z.size)
    t = temperature if temperature > 0 else 1.0
    with np.errstate(invalid="ignore"):
        x = np.where(z == m, 0.0, (z - m) / t)
    w = np.exp(x)
    order = np.argsort(-x, kind="stable")
    n = z.size
    if temperature <= 0:
        n = 1
    elif 0 < top_k < n:
        n = top_k
    s = w[order]
    if top_p < 1.0:
        total = s[:n].sum()
        before = np.concatenate(([0.0], np.cumsum(s[:n])[:-1]))
        n = max(1, int((before < top_p * total).sum()))
    if min_p > 0.0:
        n = max(1, min(n, int((s >= min_p).sum())))
    out = np.zeros_like(w)
    out[order[:n]] = s[:n]
    return out, order


def draw(weights, u):
    """First token, by index, whose cumulative weight exceeds u of the whole; -1 if none is left."""
    c = np.cumsum(weights)
    if c.size == 0 or c[-1] <= 0.0:
        return -1
    return int(min(np.searchsorted(c, u * c[-1], side="right"), np.nonzero(weights)[0][-1]))
