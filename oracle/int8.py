"""Plain CPU definition of the int8 linear and of the gradients around it.

TEST INFRASTRUCTURE ONLY (like the rest of ``oracle/``): imported by the
tests, never by the library.  It shares no code, table or constant with the
CUDA path.

Source: the quantization tutorial's symmetric per-channel formula ("How
quantization works") applied to each token of x with max_int = 127:

* sx_m = fl32(max_k |x_mk| / 127), an IEEE fp32 division; a zero token takes
  fl32(1 / 127); a token with an infinity or NaN takes NaN and codes 0;
* xq_mk = clamp(rint_half_even(fl32(x_mk / sx_m)), -127, 127);
* y_mn = bf16(s_n * sx_m * sum_k xq_mk * q_nk), the sum exact;
* dx_mk = bf16(sum_n dy_mn * s_n * q_nk), dW_nk = sum_m dy_mn * sx_m * xq_mk:
  the gradients of y = x_hat w_hat^T with respect to its factors.

Bounds are derived from the roundings of each path: u = 2^-8 is half a step
of bf16, 2^-23 one addition of an fp32 sum (twice half a step: tensor cores
may truncate).
"""
from __future__ import annotations

import numpy as np

Q8 = 127
U_BF16 = 2.0 ** -8
U_ADD = 2.0 ** -23
TINY = 2.0 ** -133            # smallest positive bf16


def quantize_x_int8(x):
    """(codes int32 [M, K], sx float32 [M]) for bf16-valued float32 x."""
    x = np.asarray(x, dtype=np.float32)
    if x.ndim != 2:
        raise TypeError("x must be 2-D")
    ok = np.isfinite(x).all(axis=1)
    xf = np.where(ok[:, None], x, np.float32(0))
    amax = np.max(np.abs(xf), axis=1).astype(np.float32)
    with np.errstate(under="ignore"):
        sx = np.where(amax == 0, np.float32(1.0), amax) / np.float32(Q8)
        t = (xf / sx[:, None]).astype(np.float32)
    codes = np.clip(np.rint(t), -Q8, Q8).astype(np.int32)
    return codes, np.where(ok, sx, np.float32(np.nan)).astype(np.float32)


def pack_rows_int8(codes):
    """Codes as canonical 8-bit rows: uint8 [M, 16 * ceil(K / 16)]."""
    M, K = codes.shape
    out = np.zeros((M, (K + 15) // 16 * 16), dtype=np.uint8)
    out[:, :K] = codes.astype(np.int8).view(np.uint8)
    return out


def qlinear_int8_ref(codes, sx, q, s):
    """(y_ref, bound) in fp64: the exact sum, three fp32 roundings (the sum's
    conversion and two products) and the bf16 rounding."""
    acc = codes.astype(np.float64) @ np.asarray(q, np.float64).T     # whole numbers below 2^53: exact
    y = acc * np.asarray(s, np.float64)[None, :] * np.asarray(sx, np.float64)[:, None]
    return y, np.abs(y) * (U_BF16 + 4 * 2.0 ** -24) + TINY


def grad_x_ref(dy, q, s):
    """(dx_ref, bound): the weight operand rounded to bf16, fp32 sums, the
    bf16 result."""
    w = np.asarray(q, np.float64) * np.asarray(s, np.float64)[:, None]
    dy = np.asarray(dy, np.float64)
    dx = dy @ w
    mag = np.abs(dy) @ np.abs(w)
    return dx, mag * (U_BF16 + dy.shape[1] * U_ADD) + np.abs(dx) * U_BF16 + TINY


def grad_w_ref(dy, codes, sx, fp32: bool):
    """(dW_ref, bound): the activation operand as one bf16 value (bf16
    result) or as three that make up its fp32 value (fp32 result), fp32 sums."""
    x = codes.astype(np.float64) * np.asarray(sx, np.float64)[:, None]
    dy = np.asarray(dy, np.float64)
    dw = dy.T @ x
    mag = np.abs(dy).T @ np.abs(x)
    if fp32:
        return dw, mag * (U_BF16 ** 3 + (3 * dy.shape[0] + 2) * U_ADD) + 1e-42
    return dw, mag * (U_BF16 + dy.shape[0] * U_ADD) + np.abs(dw) * U_BF16 + TINY
