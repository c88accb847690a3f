"""e4m3 quantisation with one fp32 scale per block of 128, the products of such matrices in fp64, and the
gradients of the MoE steps that move rows (test infrastructure only).

The sources quantise to 4 bits; this is the 8-bit counterpart, defined here: a block with largest magnitude
amax (taken as at least 2^-100) has scale s = fl(amax / 448) and codes e4m3(fl(x * fl(448 / amax))), every
step one fp32 operation rounded to nearest even.  A block that holds an infinity or a NaN has a scale or
codes that give no finite value.
"""
from __future__ import annotations

import numpy as np

from . import formats

F32 = np.float32
TINY = F32(2.0 ** -100)


def encode(y) -> np.ndarray:
    """fp32 -> e4m3fn code (uint8), RNE, saturating at 448; NaN -> 0x7F (either sign)."""
    y = np.asarray(y, dtype=F32)
    nan = np.isnan(y)
    mag = formats.e4m3_encode(np.where(nan, F32(0), np.abs(y)))
    return np.where(nan, 0x7F, mag | np.where(np.signbit(y), 0x80, 0).astype(np.uint8)).astype(np.uint8)


def _scaled(blocks, axes):
    """(codes, scales) of blocks along `axes` (kept as ones in the scales)."""
    b = np.asarray(blocks, dtype=F32)
    mag = np.abs(b)
    amax = np.max(mag, axis=axes, keepdims=True)          # NaN where the block holds one
    amax = np.where(amax < TINY, TINY, amax).astype(F32)
    with np.errstate(all="ignore"):
        s = (amax / F32(448.0)).astype(F32)
        f = (F32(448.0) / amax).astype(F32)
        return encode((b * f).astype(F32)), s


def _padded(x, rows, cols):
    m, k = x.shape
    return np.pad(np.asarray(x, dtype=F32), ((0, -m % rows), (0, -k % cols)))


def quantize_rows(x):
    """[m, k] -> codes [m, k], scales [ceil(k/128), m]."""
    m, k = x.shape
    q, s = _scaled(_padded(x, 1, 128).reshape(m, -1, 128), 2)
    return np.ascontiguousarray(q.reshape(m, -1)[:, :k]), np.ascontiguousarray(s[:, :, 0].T)


def padded_place(row_offsets, rows):
    """(column of each row, columns) of a matrix whose experts begin at multiples of 128; without offsets
    the rows follow each other."""
    if row_offsets is None:
        return np.arange(rows), -(-rows // 128) * 128
    place, at = [], 0
    for e in range(len(row_offsets) - 1):
        n = int(row_offsets[e + 1] - row_offsets[e])
        place.append(at + np.arange(n))
        at += -(-n // 128) * 128
    return np.concatenate(place), -(-rows // 128) * 128 + 128 * (len(row_offsets) - 1)


def quantize_columns(x, row_offsets=None):
    """[m, k] -> transposed codes [k, P], scales [P/128, k]; each expert's rows begin at a multiple of 128."""
    m, k = x.shape
    place, p = padded_place(row_offsets, m)
    wide = np.zeros((p, k), dtype=F32)
    wide[place] = np.asarray(x, dtype=F32)[: len(place)]
    q, s = _scaled(wide.reshape(-1, 128, k), 1)
    return np.ascontiguousarray(q.reshape(p, k).T), np.ascontiguousarray(s[:, 0])


def quantize_blocks(w):
    """[n, k] -> codes [n, k], scales [ceil(n/128), ceil(k/128)]."""
    n, k = w.shape
    b = _padded(w, 128, 128)
    q, s = _scaled(b.reshape(b.shape[0] // 128, 128, b.shape[1] // 128, 128), (1, 3))
    return np.ascontiguousarray(q.reshape(b.shape)[:n, :k]), np.ascontiguousarray(s[:, 0, :, 0])


def rows_value(q, s) -> np.ndarray:
    """fp64 values of codes with one scale per row and 128 columns."""
    return formats.e4m3_decode(q) * np.repeat(s.astype(np.float64).T, 128, axis=1)[:, : q.shape[1]]


def blocks_value(q, s) -> np.ndarray:
    """fp64 values of codes with one scale per 128 x 128 block."""
    n, k = q.shape
    return formats.e4m3_decode(q) * np.repeat(np.repeat(s.astype(np.float64), 128, 0)[:n], 128, 1)[:, :k]


def product_slack(k: int) -> float:
    """How far fp32 sums over k may be off, relative to the sum of the products' magnitudes.  The products of
    two codes are exact in fp32.  A block's 128 are summed with one rounding each, counted as a truncation
    (2^-23); its sum takes two or three fp32 roundings to scale and add (2^-24 each), and each later block one."""
    return 128 * 2.0 ** -23 + (-(-k // 128) + 3) * 2.0 ** -24


def combine_grad(dout, y, pos, w):
    """Gradients of out[t] = sum_j w[t, j] y[pos[t, j]] in fp64: (dy, dw); entries of pos < 0 are absent."""
    dout, y, w = (np.asarray(v, dtype=np.float64) for v in (dout, y, w))
    dy, dw = np.zeros_like(y), np.zeros(pos.shape)
    for t in range(pos.shape[0]):
        for j in range(pos.shape[1]):
            if pos[t, j] >= 0:
                dy[pos[t, j]] += w[t, j] * dout[t]
                dw[t, j] = dout[t] @ y[pos[t, j]]
    return dy, dw


def gather_grad(dxs, pos):
    """Gradient of xs[pos[t, j]] = x[t] in fp64."""
    dxs = np.asarray(dxs, dtype=np.float64)
    return np.stack([sum((dxs[p] for p in row if p >= 0), np.zeros(dxs.shape[1])) for row in pos]) if len(pos) else np.zeros((0, dxs.shape[1]))
