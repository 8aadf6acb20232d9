"""The int8 linear and the gradients at the ends of the number range and of
their arguments: scales far from one, many tokens through few rows, infinite
gradients, the accuracy of long fp32 sums, contradictory arguments."""
import numpy as np
import pytest

import oracle
import workloads

pytestmark = pytest.mark.gpu

U_SUB = 2.0 ** -134           # half of bf16's smallest step


@pytest.fixture(scope="module")
def mpw():
    import mixed_precision_weight_row_b200 as m

    return m


def _torch():
    import torch

    return torch


def _w(N, K, seed):
    return np.random.default_rng(seed).standard_normal((N, K)).astype(np.float32) * np.float32(0.02)


def _rows(mpw, W, b, layout="canonical"):
    torch = _torch()
    packed, scales = mpw.quantize_pack(torch.from_numpy(W).cuda(), b)
    if layout != "canonical":
        packed = mpw.repack(packed, W.shape[1], b, "canonical", layout)
    return packed, scales


def _inside(got, ref, bound, what):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of bound, first at {np.argwhere(bad)[:3].tolist()}"


def _same(got, want, what):
    """Equal infinities and NaNs where the definition has them."""
    got = got.double().cpu().numpy()
    for f in (np.isnan, np.isposinf, np.isneginf):
        assert np.array_equal(f(got), f(want)), what


# ---- scales -----------------------------------------------------------------

TINY_SCALES = [4e-41, 6e-40, 1e-39, 7e-39, 1.2e-38, 3e-38, 1e-37, 1e-36, 1e-35, 1e-33]


@pytest.mark.parametrize("layout", ["canonical", "paired"])
@pytest.mark.parametrize("M", [40, 300, 800])
@pytest.mark.parametrize("b", [4, 6, 8, 9, 12])
def test_grad_x_tiny_scales(mpw, b, M, layout):
    """A weight operand w = s q is off by at most half a step of bf16: 2^-8 of
    it, or 2^-134 below bf16's normal numbers."""
    torch = _torch()
    N, K = 70, 96
    W = _w(N, K, b)
    packed, _ = _rows(mpw, W, b, layout)
    q, _ = oracle.quantize(W, b)
    s = np.array([TINY_SCALES[n % len(TINY_SCALES)] for n in range(N)], np.float32)
    dy = (torch.randn((M, N), generator=torch.Generator().manual_seed(M)) * 1e34).to(torch.bfloat16)
    # rows of very different scales, each alone against its own bound
    for part in range(len(TINY_SCALES)):
        d = torch.zeros_like(dy)
        d[:, part::len(TINY_SCALES)] = dy[:, part::len(TINY_SCALES)]
        dx = mpw.qlinear_grad_x(d.cuda(), packed, torch.from_numpy(s).cuda(), b, K, layout=layout)
        ref, bound = oracle.grad_x_ref(d.float().numpy(), q, s)
        bound = bound + (np.abs(d.double().numpy()).sum(1) * U_SUB)[:, None]
        _inside(dx, ref, bound, f"b={b} {layout} M={M} s={TINY_SCALES[part]}")


@pytest.mark.parametrize("M", [40, 800])
@pytest.mark.parametrize("b", [4, 6, 8, 9, 12])
def test_grad_x_largest_scales(mpw, b, M):
    """Zero codes stay zeros under the largest finite scales, and codes whose
    product with them is finite keep it."""
    torch = _torch()
    N, K = 24, 64
    W = _w(N, K, b)
    W[3] = 0
    W[7] = 0
    packed, scales = _rows(mpw, W, b)
    dy = (torch.randn((M, N), generator=torch.Generator().manual_seed(M)) * 1e-3).to(torch.bfloat16).cuda()
    want = mpw.qlinear_grad_x(dy, packed, scales, b, K)
    scales[3], scales[7] = 3.4028234e38, 3.395e38
    assert torch.equal(mpw.qlinear_grad_x(dy, packed, scales, b, K), want)
    q, s = oracle.quantize(W, b)
    s = s.copy()
    s[5] = np.float32(3e38 / 2 ** (b - 1))
    scales[3], scales[7], scales[5] = 1.0, 1.0, float(s[5])
    dy = dy * 1e-3
    dx = mpw.qlinear_grad_x(dy, packed, scales, b, K)
    ref, bound = oracle.grad_x_ref(dy.float().cpu().numpy(), q, s)
    _inside(dx, ref, bound, f"b={b} M={M}")


@pytest.mark.parametrize("M", [1, 2, 4, 40, 300, 1100])
@pytest.mark.parametrize("b", [4, 6, 8])
def test_qlinear_int8_scales_apart(mpw, b, M):
    """Large weights with small tokens and the reverse: the result is finite
    and normal, so no product on the way to it may overflow or lose bits."""
    torch = _torch()
    N, K = 40, 160
    W = _w(N, K, 1)
    q, _ = oracle.quantize(W, b)
    packed, _ = _rows(mpw, W, b)
    x = workloads.gen_x(M, K, 3)
    codes, _ = oracle.quantize_x_int8(x.float().numpy())
    xq, _ = mpw.quantize_x_int8(x.cuda())
    for s_w, s_x in [(3e36, 1e-37), (4.8e37, 3e-40), (1e-38, 1e36), (2e-43, 1e36), (1e30, 1e-30), (1e-30, 1e30),
                     (1e-20, 1e-19)]:
        s, sx = np.full(N, s_w, np.float32), np.full(M, s_x, np.float32)
        y = mpw.qlinear_int8(None, packed, torch.from_numpy(s).cuda(), b, xq=xq, sx=torch.from_numpy(sx).cuda(), K=K)
        ref, bound = oracle.qlinear_int8_ref(codes, sx, q, s)
        _inside(y, ref, bound, f"b={b} M={M} s={s_w} sx={s_x}")


# ---- narrow outputs -------------------------------------------------------------


@pytest.mark.parametrize("layout", ["canonical", "paired"])
@pytest.mark.parametrize("N,K,M,b", [(40, 17408, 193, 8), (256, 2048, 700, 8), (256, 5120, 1025, 6), (130, 1024, 3001, 4),
                                     (33, 96, 2000, 7), (1000, 512, 1030, 5), (16, 4096, 8192, 6), (16, 4096, 8193, 8)])
def test_qlinear_int8_narrow_outputs(mpw, N, K, M, b, layout):
    """Many tokens through few rows, on either side of the border between the
    kernels: the exact sums."""
    torch = _torch()
    W = _w(N, K, N)
    packed, scales = _rows(mpw, W, b, layout)
    x = workloads.gen_x(M, K, M)
    y = mpw.qlinear_int8(x.cuda(), packed, scales, b, layout=layout)
    pick = np.unique(np.concatenate([[0, M - 1], np.random.default_rng(M).integers(0, M, 200)]))
    q, s = oracle.quantize(W, b)
    codes, sx = oracle.quantize_x_int8(x[torch.from_numpy(pick)].float().numpy())
    ref, bound = oracle.qlinear_int8_ref(codes, sx, q, s)
    _inside(y[torch.from_numpy(pick).cuda()], ref, bound, f"b={b} {layout} M={M} N={N} K={K}")
    assert mpw.device_error() == 0


def test_narrow_outputs_share_k(mpw):
    """A product of few tiles runs where several SMs share a tile's K, which
    takes no workspace for expanded rows, at any number of tokens that leaves
    it few tiles; one of many tiles does not."""
    f = mpw.lib.mpw_qlinear_int8_workspace_bytes
    for M, N, K in [(1024, 256, 17408), (1025, 256, 17408), (4096, 256, 17408), (8192, 128, 17408), (2000, 512, 5120)]:
        assert f(6, 0, M, N, K) == 0, (M, N, K)
    for M, N, K in [(8193, 256, 17408), (1025, 17408, 5120), (1280, 4096, 4096)]:
        assert f(6, 0, M, N, K) >= N * K, (M, N, K)


# ---- infinite gradients -------------------------------------------------------


@pytest.mark.parametrize("M,N,K", [(5, 40, 64), (16, 64, 128), (300, 130, 100), (1100, 257, 333), (4100, 300, 72)])
@pytest.mark.parametrize("fp32", [False, True])
def test_infinite_dy(mpw, M, N, K, fp32):
    """inf times a nonzero code is an infinity, inf times a zero code NaN."""
    torch = _torch()
    x = workloads.gen_x(M, K, M)
    x[1] = 0
    x[2, :7] = torch.tensor([127.0, 64.0, -32.0, 1.0, -1.0, 3.0, 0.0])     # codes of a scale of 1: few bits each
    x[2, 7:] = 5.0
    x[3, ::3] = 0
    xq, sx = mpw.quantize_x_int8(x.cuda())
    dy = (torch.randn((M, N), generator=torch.Generator().manual_seed(1)) * 1e-3).to(torch.bfloat16)
    clean = mpw.qlinear_grad_w_int8(dy.cuda(), xq, sx, K, dtype=torch.float32 if fp32 else torch.bfloat16)
    inf = float("inf")
    dy[2, 0], dy[3, 1], dy[M - 1, 2], dy[0, 4], dy[M - 1, 4] = inf, -inf, inf, inf, -inf
    dy[1, 5] = inf
    dW = mpw.qlinear_grad_w_int8(dy.cuda(), xq, sx, K, dtype=torch.float32 if fp32 else torch.bfloat16)
    codes, sxr = oracle.quantize_x_int8(x.float().numpy())
    xh = codes.astype(np.float64) * sxr.astype(np.float64)[:, None]
    with np.errstate(invalid="ignore"):
        want = (dy.double().numpy().T[:, :, None][:8] * xh[None]).sum(1)
    _same(dW[:8], want, f"fp32={fp32} M={M} N={N} K={K}")
    for n in (3, 6, 7):
        assert torch.equal(dW[n], clean[n])
    assert torch.equal(dW[8:], clean[8:])


# ---- long fp32 sums -------------------------------------------------------------


@pytest.mark.parametrize("M,N,K", [(1000, 300, 512), (2048, 256, 512), (8200, 130, 512), (8192, 2600, 1280)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_w_fp32_sums(mpw, M, N, K, accumulate):
    """A sum of at most 768 tokens in one go, the rest added to nearest: within
    1e-6 of the norm for operands of mean zero, 1.6e-6 for operands of one
    sign, at any of these lengths.  (All tokens in one go are off by 2.1e-6 and
    5.6e-6 at 2048 tokens, 9e-6 and 35e-6 at 8192.)"""
    torch = _torch()
    x = workloads.gen_x(M, K, 1).cuda()
    dy = (torch.randn((M, N), generator=torch.Generator().manual_seed(2)) * 1e-3).to(torch.bfloat16).cuda()
    for x, dy, limit in ((x, dy, 1e-6), (x.abs(), dy.abs(), 1.6e-6)):
        xq, sx = mpw.quantize_x_int8(x)
        dW = torch.zeros((N, K), device="cuda")
        mpw.qlinear_grad_w_int8(dy, xq, sx, K, dW=dW, accumulate=accumulate)
        xh = mpw.unpack(xq, K, 8).double() * sx.double()[:, None]
        ref = dy.double().T @ xh
        assert float((dW.double() - ref).norm() / ref.norm()) <= limit


# ---- arguments ------------------------------------------------------------------


def test_contradictory_arguments_are_refused(mpw):
    torch = _torch()
    M, N, K = 20, 24, 64
    packed, scales = _rows(mpw, _w(N, K, 1), 6)
    x = workloads.gen_x(M, K, 1).cuda()
    xq, sx = mpw.quantize_x_int8(x)
    want = mpw.qlinear_int8(x, packed, scales, 6)
    for kw in (dict(xq=xq, sx=sx), dict(xq=xq, sx=sx, K=K), dict(K=K)):
        assert torch.equal(mpw.qlinear_int8(x, packed, scales, 6, **kw), want)
    with pytest.raises(ValueError, match="xq and sx"):
        mpw.qlinear_int8(None, packed, scales, 6, xq=xq)
    with pytest.raises(ValueError, match="xq and sx"):
        mpw.qlinear_int8(x, packed, scales, 6, sx=sx)
    with pytest.raises(ValueError, match="K is needed"):
        mpw.qlinear_int8(None, packed, scales, 6, xq=xq, sx=sx)
    with pytest.raises(ValueError, match="x must have shape"):
        mpw.qlinear_int8(x[1:], packed, scales, 6, xq=xq, sx=sx)
    with pytest.raises(ValueError, match="x must have shape"):
        mpw.qlinear_int8(x, packed, scales, 6, xq=xq, sx=sx, K=K - 1)
    with pytest.raises(ValueError, match="x must have shape"):
        mpw.qlinear_int8(x, packed, scales, 6, K=K - 1)
