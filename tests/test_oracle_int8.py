"""Pins of the oracle's int8 linear and gradients (oracle/int8.py) against what
the mathematics fixes:

* codes and scales against a Fraction evaluation of the formula (each quotient
  rounded to fp32 by numpy's scalar division only), ties to even, the largest
  element of a token reaching +-127, zero tokens, non-finite tokens;
* the same codes as the per-row quantizer at b = 8 gives for the same matrix;
* the linear against a triple loop on whole numbers;
* the gradients against central differences of the product;
* planted mistakes (ties away from zero, truncation, max_int 128, one scale
  for the whole tensor, a dropped token scale) each fail a pin.
"""
from fractions import Fraction

import numpy as np
import pytest

import oracle
from oracle import int8 as oi


def _bf16(a):
    a = np.ascontiguousarray(a, dtype=np.float32)
    u = a.view(np.uint32)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)


def _x(M, K, seed):
    x = _bf16(np.random.default_rng(seed).standard_normal((M, K)) * 3)
    if M > 2:
        x[1] = 0
        x[2] = _bf16(x[2] * 1e-36)
    return x


def _codes_by_fractions(x):
    out = np.zeros(x.shape, np.int64)
    for m, row in enumerate(x):
        top = max(abs(float(v)) for v in row) or 1.0
        s = np.float32(np.float32(top) / np.float32(127))
        for k, v in enumerate(row):
            t = Fraction(float(np.float32(v / s)))
            lo = t.numerator // t.denominator
            frac = t - lo
            out[m, k] = lo + (1 if frac > Fraction(1, 2) or (frac == Fraction(1, 2) and lo % 2) else 0)
    return np.clip(out, -127, 127)


def check_codes(fn):
    for M, K, seed in [(1, 1, 0), (4, 9, 1), (5, 40, 2)]:
        x = _x(M, K, seed)
        codes, sx = fn(x)
        assert np.array_equal(codes, _codes_by_fractions(x))
        nz = np.any(x != 0, axis=1)
        assert np.all(np.abs(codes).max(axis=1)[nz] == 127)
        assert np.all(codes[~nz] == 0) and np.all(sx[~nz] == np.float32(1) / np.float32(127))
        # every element within half a step (and the quotient's own rounding) of what its code stands for
        err = np.abs(codes * sx.astype(np.float64)[:, None] - x)
        assert np.all(err <= sx.astype(np.float64)[:, None] * (0.5 + 127 * 2.0 ** -22))
    # exact ties: scale 1, quotients k + 1/2
    x = np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5]], np.float32)
    assert fn(x)[0].tolist() == [[127, 0, 2, 2, 0, -2, -2]]


def test_codes():
    check_codes(oi.quantize_x_int8)


def test_same_as_the_row_quantizer_at_eight_bits():
    x = _x(6, 50, 5)
    codes, sx = oi.quantize_x_int8(x)
    q, s = oracle.quantize(x, 8)
    assert np.array_equal(codes, q) and np.array_equal(sx.view(np.uint32), s.view(np.uint32))
    assert np.array_equal(oi.pack_rows_int8(codes), oracle.quantize_pack(x, 8)[0])


def test_non_finite_token():
    x = _x(5, 12, 6)
    x[3, 4] = np.inf
    x[4, 0] = np.nan
    codes, sx = oi.quantize_x_int8(x)
    assert np.isnan(sx[3:]).all() and (codes[3:] == 0).all()
    keep, kept = oi.quantize_x_int8(x[:3])
    assert np.array_equal(codes[:3], keep) and np.array_equal(sx[:3], kept)


def check_linear(ref):
    rng = np.random.default_rng(7)
    codes = rng.integers(-127, 128, (3, 11))
    q = rng.integers(-31, 32, (4, 11))
    sx = rng.random(3).astype(np.float32)
    s = rng.random(4).astype(np.float32)
    y, bound = ref(codes, sx, q, s)
    for m in range(3):
        for n in range(4):
            want = sum(int(codes[m, k]) * int(q[n, k]) for k in range(11)) * Fraction(float(s[n])) * Fraction(float(sx[m]))
            assert abs(Fraction(float(y[m, n])) - want) <= abs(want) * Fraction(1, 2 ** 50)
            assert abs(float(want)) * 2.0 ** -8 <= bound[m, n] <= abs(float(want)) * 2.0 ** -7 + 1e-30


def test_linear():
    check_linear(oi.qlinear_int8_ref)


def test_gradients_are_the_differences_of_the_product():
    rng = np.random.default_rng(8)
    M, N, K = 5, 4, 7
    codes = rng.integers(-127, 128, (M, K))
    q = rng.integers(-7, 8, (N, K))
    sx, s = rng.random(M).astype(np.float32), rng.random(N).astype(np.float32)
    dy = rng.standard_normal((M, N))
    x, w = codes * sx.astype(np.float64)[:, None], q * s.astype(np.float64)[:, None]

    def loss(a, b):
        return float(np.sum(dy * (a @ b.T)))

    dx, _ = oi.grad_x_ref(dy, q, s)
    dw, _ = oi.grad_w_ref(dy, codes, sx, True)
    h = 2.0 ** -10
    for i, j in [(0, 0), (2, 3), (4, 6)]:
        e = np.zeros_like(x)
        e[i, j] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i, j]) < 1e-8
    for i, j in [(0, 0), (1, 5), (3, 6)]:
        e = np.zeros_like(w)
        e[i, j] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i, j]) < 1e-6


def _mutant(top=127.0, rnd=np.rint, whole=False):
    def fn(x):
        amax = np.abs(x).max(axis=1)
        if whole:
            amax = np.full_like(amax, np.abs(x).max())
        sx = (np.where(amax == 0, 1, amax) / np.float32(top)).astype(np.float32)
        return np.clip(rnd((x / sx[:, None]).astype(np.float32)), -127, 127).astype(np.int32), sx
    return fn


@pytest.mark.parametrize("fn", [
    _mutant(rnd=lambda t: np.sign(t) * np.floor(np.abs(t) + 0.5)),
    _mutant(rnd=np.trunc),
    _mutant(top=128.0),
    _mutant(whole=True),
], ids=["ties-away", "truncation", "max-int-128", "one-scale"])
def test_planted_mistakes_in_the_codes(fn):
    with pytest.raises(AssertionError):
        check_codes(fn)


def test_planted_mistake_in_the_linear():
    with pytest.raises(AssertionError):
        check_linear(lambda codes, sx, q, s: oi.qlinear_int8_ref(codes, np.ones_like(sx), q, s))
