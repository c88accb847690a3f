"""Further pins for oracle/fp8.py: scales, factors and codes against exact rationals, the values of codes and the product
of two quantised matrices against loops, and the helpers of the GPU tests against the same."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import test_gpu_fp8
import test_gpu_fp8_edges
import test_gpu_fp8_range
from oracle import fp8
from oracle.formats import e4m3_decode

F32 = np.float32


def nearest(v: Fraction, bits: int, least: int) -> Fraction:
    """v to `bits` significant bits, no step below 2^least, ties to even."""
    if v == 0:
        return v
    e = 0
    while Fraction(2) ** (e + 1) <= abs(v):
        e += 1
    while Fraction(2) ** e > abs(v):
        e -= 1
    step = Fraction(2) ** max(e - bits + 1, least)
    n, rest = divmod(v, step)
    up = rest * 2 > step or (rest * 2 == step and n % 2 == 1)
    return (n + 1 if up else n) * step


def fp32(v: Fraction) -> Fraction:
    return nearest(v, 24, -149)


def exact(x) -> Fraction:
    return Fraction(float(x))


def test_scales_and_codes_against_rationals():
    """s = fl(amax / 448), code = e4m3(fl(x * fl(448 / amax))), clamped to 448, every fl one rounding to nearest even."""
    r = np.random.default_rng(0)
    x = (r.standard_normal((12, 128)) * np.exp2(r.integers(-12, 3, (12, 128)))).astype(F32)
    x[1] *= F32(2.0 ** -90)
    x[2] = 0
    x[3] *= F32(2.0 ** 100)
    x[4, :] = F32(2.0 ** -120)                              # below the least magnitude that a scale is taken from
    x[5, 0], x[5, 1:] = F32(448.0), np.linspace(17.0, 19.0, 127).astype(F32)     # a step of 2 there: ties among them
    q, s = fp8.quantize_rows(x)
    v = e4m3_decode(q)
    for i in range(len(x)):
        amax = max(max(abs(exact(t)) for t in x[i]), Fraction(2) ** -100)
        assert exact(s[0, i]) == fp32(amax / 448)
        factor = fp32(448 / amax)
        for j in range(128):
            y = fp32(exact(x[i, j]) * factor)
            assert exact(v[i, j]) == max(min(nearest(y, 4, -9), Fraction(448)), Fraction(-448)), (i, j)


def matrices():
    r = np.random.default_rng(1)
    x = (r.standard_normal((5, 272)) * np.exp2(r.integers(-6, 7, (5, 1)))).astype(F32)
    w = (r.standard_normal((140, 272)) * 0.02).astype(F32)
    return x, w


def test_values_against_loops():
    x, w = matrices()
    q, s = fp8.quantize_rows(x)
    v = fp8.rows_value(q, s)
    for i in range(5):
        for k in range(272):
            assert v[i, k] == float(e4m3_decode(q[i, k])) * float(s[k // 128, i])
    q, s = fp8.quantize_blocks(w)
    v = fp8.blocks_value(q, s)
    for i in (0, 127, 128, 139):
        for k in range(272):
            assert v[i, k] == float(e4m3_decode(q[i, k])) * float(s[i // 128, k // 128])


def test_products_against_loops():
    """D[i, j] = sum over blocks of sa sb times the block's sum, in exact rationals, against the fp64 product of the values."""
    x, w = matrices()
    qa, sa = fp8.quantize_rows(x)
    for (qb, sb), scale, value in ((fp8.quantize_blocks(w), lambda s, j, b: s[j // 128, b], fp8.blocks_value),
                                   (fp8.quantize_rows(w), lambda s, j, b: s[b, j], fp8.rows_value)):
        a, b = fp8.rows_value(qa, sa), value(qb, sb)
        got, size = a @ b.T, np.abs(a) @ np.abs(b).T
        ca, cb = e4m3_decode(qa), e4m3_decode(qb)
        for i, j in ((0, 0), (1, 5), (2, 127), (3, 128), (4, 139)):
            want = Fraction(0)
            for block in range(3):
                part = sum((exact(ca[i, k]) * exact(cb[j, k]) for k in range(128 * block, min(272, 128 * block + 128))), Fraction(0))
                want += exact(sa[block, i]) * exact(scale(sb, j, block)) * part
            # (the values are exact: 4 + 24 bits; 272 products and their sums, each rounded once in fp64)
            assert abs(exact(got[i, j]) - want) <= Fraction(2) ** -52 * 280 * exact(size[i, j])


@pytest.mark.parametrize("helpers", [test_gpu_fp8, test_gpu_fp8_edges, test_gpu_fp8_range])
def test_helpers_of_the_gpu_tests(helpers):
    x, w = matrices()

    def tensors(q, s):
        return torch.from_numpy(q).view(torch.float8_e4m3fn), torch.from_numpy(s)

    for m, quantise, value, helper in ((x, fp8.quantize_rows, fp8.rows_value, helpers.rows64), (w, fp8.quantize_blocks, fp8.blocks_value, helpers.blocks64)):
        q, s = quantise(m)
        assert np.array_equal(helper(*tensors(q, s)).numpy(), value(q, s))
