"""The int8 linear and the gradients of packed linears against the oracle's
fp64 definitions (oracle/int8.py), with the bounds derived there.

* mpw_quantize_x_int8: scales (bit patterns), every code and the zero padding,
  for odd K, misaligned rows, zero, tiny, infinite and NaN tokens.
* mpw_qlinear_int8: every width and layout from one token to several tiles,
  ragged M, N and K, the largest sums, full prefill shapes on sampled rows.
* rows, tokens and results whose offsets pass 32 bits.
* gradients: every width, both result types, accumulation, odd sizes, the
  differences of the product.
* together: a two-layer step with gradients, accumulated weight gradients to
  the allocator's sensitivities, captured graphs, other streams, two calls
  at once, untouched memory around the results, refusals.
"""
import numpy as np
import pytest

import oracle
import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mpw():
    import mixed_precision_weight_row_b200 as m

    return m


def _torch():
    import torch

    return torch


def _x(M, K, seed):
    torch = _torch()
    x = workloads.gen_x(M, K, seed)
    if M > 3:
        x[1] = 0                                      # a zero token
        x[2] = x[2] * 1e-37                           # a subnormal scale
        x[3, :5] = torch.tensor([200.0, -3.0, 0.5, 1e-30, -200.0])[:min(5, K)].to(torch.bfloat16) if K >= 5 else 1.0
    return x


def _w(N, K, seed):
    W = np.random.default_rng(seed).standard_normal((N, K)).astype(np.float32) * np.float32(0.02)
    W[min(5, N - 1)] = 0
    return W


def _dy(M, N, seed):
    torch = _torch()
    return (torch.randn((M, N), generator=torch.Generator().manual_seed(seed)) * 1e-3).to(torch.bfloat16)


def _rows(mpw, W, b, layout):
    torch = _torch()
    packed, scales = mpw.quantize_pack(torch.from_numpy(W).cuda(), b)
    if layout != "canonical":
        packed = mpw.repack(packed, W.shape[1], b, "canonical", layout)
    return packed, scales


def _guarded(shape, dtype, fill):
    """A tensor inside a larger buffer whose surroundings are checked."""
    torch = _torch()
    n = int(np.prod(shape))
    buf = torch.full((n + 256,), fill, dtype=dtype, device="cuda")
    return buf, buf[128:128 + n].view(shape)


def _intact(buf, n, fill):
    return bool((buf[:128] == fill).all() and (buf[128 + n:] == fill).all())


def _inside(got, ref, bound, what):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of bound, first at {np.argwhere(bad)[:3].tolist()}"


# ---- quantize_x_int8 --------------------------------------------------------


@pytest.mark.parametrize("M,K", [(1, 1), (1, 16), (5, 7), (4, 777), (33, 4112), (300, 5120), (7, 17408), (3, 40000),
                                 (2, 131071), (2048, 5120)])
def test_quantize_x_int8_exact(mpw, M, K):
    torch = _torch()
    x = _x(M, K, M + K)
    buf, xq = _guarded((M, mpw.packed_row_bytes(K, 8)), torch.uint8, 0xA5)
    sx = torch.full((M,), 7.0, device="cuda")
    mpw.quantize_x_int8(x.cuda(), xq=xq, sx=sx)
    codes, sx_ref = oracle.quantize_x_int8(x.float().numpy())
    assert np.array_equal(sx.cpu().numpy().view(np.uint32), sx_ref.view(np.uint32))
    assert np.array_equal(xq.cpu().numpy(), oracle.pack_rows_int8(codes))
    assert _intact(buf, xq.numel(), 0xA5)


def test_quantize_x_int8_near_ties(mpw):
    """Values whose quotient lies on or next to k + 1/2: every bf16 pattern of
    two binades against several largest values."""
    torch = _torch()
    v = (torch.arange(0x3F80, 0x4080, dtype=torch.int32) & 0xFFFF).to(torch.int16).view(torch.bfloat16)
    rows = []
    for top in (127.0, 63.5, 254.0, 126.5, 3.0, 255.0, 100.0, 97.0, 120.0, 2.0 ** -100, 2.0 ** 100):
        big = torch.tensor([top], dtype=torch.bfloat16)
        for scale in (1.0, -0.25, 16.0):
            x = (v.float() * scale * (big.float() / 127.0)).to(torch.bfloat16)
            rows.append(torch.cat([big, x, v, -v])[:1 + 3 * v.numel()])
    k = torch.arange(-126, 127).float() + 0.5                    # exact ties for a scale of 1
    n = rows[0].numel()
    tie = torch.zeros(n, dtype=torch.bfloat16)
    tie[0], tie[1:1 + k.numel()] = 127.0, k.to(torch.bfloat16)
    rows.append(tie)
    x = torch.stack(rows)
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % 8))
    codes, sx_ref = oracle.quantize_x_int8(x.float().numpy())
    for part in (x, x.repeat(200, 1)):                           # either thread count
        xq, sx = mpw.quantize_x_int8(part.cuda())
        assert np.array_equal(xq[:len(rows)].cpu().numpy(), oracle.pack_rows_int8(codes))
        assert np.array_equal(sx[:len(rows)].cpu().numpy().view(np.uint32), sx_ref.view(np.uint32))


def test_quantize_x_int8_misaligned_rows(mpw):
    torch = _torch()
    big = _x(1, 1 + 6 * 64, 3).cuda().reshape(-1)
    x = big[1:].view(6, 64)                            # 2 bytes past an aligned address
    xq, sx = mpw.quantize_x_int8(x)
    codes, sx_ref = oracle.quantize_x_int8(x.float().cpu().numpy())
    assert np.array_equal(xq.cpu().numpy(), oracle.pack_rows_int8(codes))
    assert np.array_equal(sx.cpu().numpy(), sx_ref)


def test_quantize_x_int8_is_the_row_quantizer_at_eight_bits(mpw):
    torch = _torch()
    x = _x(40, 1000, 9).cuda()
    xq, sx = mpw.quantize_x_int8(x)
    packed, scales = mpw.quantize_pack(x.float(), 8)
    assert torch.equal(xq, packed) and torch.equal(sx, scales)
    back = mpw.dequantize(xq, sx, 1000, 8)             # the checkpoint restored
    assert bool(((back - x.float()).abs() <= 0.5001 * sx[:, None]).all())


@pytest.mark.parametrize("K", [64, 77])
def test_non_finite_tokens_stay_apart(mpw, K):
    torch = _torch()
    M, N = 6, 40
    x = _x(M, K, 4)
    x[0, K - 1] = float("inf")
    x[4, 0] = float("nan")
    W = _w(N, K, 5)
    packed, scales = _rows(mpw, W, 6, "canonical")
    xq, sx = mpw.quantize_x_int8(x.cuda())
    assert torch.isnan(sx[[0, 4]]).all() and (xq[[0, 4]] == 0).all()
    y = mpw.qlinear_int8(None, packed, scales, 6, xq=xq, sx=sx, K=K)
    assert torch.isnan(y[[0, 4]]).all()
    keep = [1, 2, 3, 5]
    alone = mpw.qlinear_int8(x[keep].cuda(), packed, scales, 6)
    assert torch.equal(y[keep], alone)


# ---- qlinear_int8 -----------------------------------------------------------


def _check_linear(mpw, N, K, M, b, layout, seed=0):
    torch = _torch()
    W = _w(N, K, N + K + b)
    packed, scales = _rows(mpw, W, b, layout)
    x = _x(M, K, seed + M)
    buf, y = _guarded((M, N), torch.bfloat16, 7.0)
    mpw.qlinear_int8(x.cuda(), packed, scales, b, y=y, layout=layout)
    q, s = oracle.quantize(W, b)
    codes, sx = oracle.quantize_x_int8(x.float().numpy())
    ref, bound = oracle.qlinear_int8_ref(codes, sx, q, s)
    _inside(y, ref, bound, f"b={b} {layout} M={M} N={N} K={K}")
    assert _intact(buf, y.numel(), 7.0)


SMALL = [(1, 1, 1), (3, 5, 2), (100, 256, 1), (17, 31, 3), (128, 512, 40), (257, 1024, 300), (65, 777, 17),
         (130, 5120, 513), (1031, 333, 9), (64, 4096, 256), (48, 160, 4), (200, 129, 33)]


@pytest.mark.parametrize("b", [4, 5, 6, 7, 8])
@pytest.mark.parametrize("N,K,M", SMALL)
def test_qlinear_int8_canonical(mpw, N, K, M, b):
    _check_linear(mpw, N, K, M, b, "canonical")


@pytest.mark.parametrize("b", [4, 5, 6, 7, 8])
@pytest.mark.parametrize("N,K,M", [(1, 32, 1), (100, 256, 1), (17, 96, 3), (128, 512, 40), (257, 1024, 300),
                                   (65, 800, 17), (1031, 352, 8), (300, 5120, 2)])
def test_qlinear_int8_paired(mpw, N, K, M, b):
    _check_linear(mpw, N, K, M, b, "paired")


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 12, 16, 17, 31, 32, 33, 48, 64, 65, 96, 128, 129, 192, 200, 256, 257,
                               384, 511, 512, 513, 700, 1024])
def test_qlinear_int8_every_token_count(mpw, M):
    _check_linear(mpw, 520, 1280, M, 6, "canonical")


@pytest.mark.parametrize("layout", ["canonical", "paired"])
@pytest.mark.parametrize("b", [4, 5, 6, 7, 8])
@pytest.mark.parametrize("N,K,M", [(40, 96, 1025), (257, 1024, 1111), (600, 160, 1500)])
def test_qlinear_int8_many_tokens(mpw, N, K, M, b, layout):
    _check_linear(mpw, N, K, M, b, layout)


@pytest.mark.parametrize("M", [1, 7, 40, 300, 700, 1100])
@pytest.mark.parametrize("b", [4, 7, 8])
def test_qlinear_int8_long_rows(mpw, M, b):
    _check_linear(mpw, 72, 17408, M, b, "canonical")


@pytest.mark.parametrize("M", [1, 20, 600, 1030])
def test_qlinear_int8_largest_sums(mpw, M):
    """Every product +-127 * 127 over the longest K: the 32-bit sums hold."""
    torch = _torch()
    K, N = 131071, 24
    x = torch.ones((M, K), dtype=torch.bfloat16)
    x[M // 2] = -1
    W = np.ones((N, K), np.float32)
    W[1::2] = -1
    packed, scales = _rows(mpw, W, 8, "canonical")
    y = mpw.qlinear_int8(x.cuda(), packed, scales, 8)
    codes, sx = oracle.quantize_x_int8(x.float().numpy())
    q, s = oracle.quantize(W, 8)
    ref, bound = oracle.qlinear_int8_ref(codes, sx, q, s)
    _inside(y, ref, bound, "largest sums")


@pytest.mark.parametrize("name,M,b", [("up", 2048, 6), ("o", 2048, 8), ("up", 1, 6), ("up", 24, 5), ("o", 333, 7)])
def test_qlinear_int8_workload_sampled(mpw, name, M, b):
    torch = _torch()
    c = workloads.PREFILL
    _, N, K = [s for s in c["shapes"] if s[0] == name][0]
    Wt = workloads.gen_weight_torch(N, K, c["sigma"], 11 + N)
    rows = np.unique(np.concatenate([[0, N - 1], np.random.default_rng(N + b).choice(N, 60, replace=False)]))
    W_rows = Wt[torch.from_numpy(rows).cuda()].cpu().numpy()
    packed, scales = mpw.quantize_pack(Wt, b)
    x = workloads.gen_x(M, K, c["x_seed"])
    y = mpw.qlinear_int8(x.cuda(), packed, scales, b)
    q, s = oracle.quantize(W_rows, b)
    codes, sx = oracle.quantize_x_int8(x.float().numpy())
    ref, bound = oracle.qlinear_int8_ref(codes, sx, q, s)
    _inside(y[:, torch.from_numpy(rows).cuda()], ref, bound, name)
    assert mpw.device_error() == 0


@pytest.mark.parametrize("M", [1, 20, 1100])
def test_qlinear_int8_rows_past_32_bits(mpw, M):
    """2.4 GB of rows, 4.8 G codes: a block of rows again and again, so that every block's results are the same."""
    torch = _torch()
    rows, times, K, b = 4096, 72, 16384, 4
    block, scales = mpw.quantize_pack(workloads.gen_weight_torch(rows, K, 0.02, 5), b)
    xq, sx = mpw.quantize_x_int8(workloads.gen_x(M, K, 6).cuda())
    ref = mpw.qlinear_int8(None, block, scales, b, xq=xq, sx=sx, K=K)
    y = mpw.qlinear_int8(None, block.repeat(times, 1), scales.repeat(times), b, xq=xq, sx=sx, K=K)
    assert torch.equal(y.view(M, times, rows), ref[:, None].expand(-1, times, -1))
    assert mpw.device_error() == 0


def test_tokens_past_32_bits(mpw):
    """4.9 G activations, then 4.4 G results and their gradients: tokens again
    and again.  Of dy only the last token, or the last column, is not zero:
    every sum is one product, whatever the order."""
    torch = _torch()
    tokens, times, K = 1000, 300, 16384
    x = workloads.gen_x(tokens, K, 7).cuda()
    xq, sx = mpw.quantize_x_int8(x)
    xq2, sx2 = mpw.quantize_x_int8(x.repeat(times, 1))
    assert torch.equal(sx2.view(times, tokens), sx.expand(times, -1))
    for t in range(times):
        assert torch.equal(xq2[t * tokens:(t + 1) * tokens], xq)
    del x, xq2, sx2

    times, N, K, b = 110, 40000, 64, 6
    M = tokens * times
    packed, scales = mpw.quantize_pack(workloads.gen_weight_torch(N, K, 0.02, 8), b)
    xq, sx = mpw.quantize_x_int8(workloads.gen_x(tokens, K, 9).cuda())
    xq2, sx2 = xq.repeat(times, 1), sx.repeat(times)
    ref = mpw.qlinear_int8(None, packed, scales, b, xq=xq, sx=sx, K=K)
    y = mpw.qlinear_int8(None, packed, scales, b, xq=xq2, sx=sx2, K=K)
    for t in range(times):
        assert torch.equal(y[t * tokens:(t + 1) * tokens], ref)
    dy = y.zero_()
    dy[:, -1] = torch.arange(M, device="cuda") % 251 - 125
    dx = mpw.qlinear_grad_x(dy, packed, scales, b, K)
    one = mpw.qlinear_grad_x(dy[:1000, -8:].contiguous(), packed[-8:], scales[-8:], b, K)
    assert torch.equal(dx[:1000], one)
    assert torch.equal(dx[-1000:], mpw.qlinear_grad_x(dy[-1000:, -8:].contiguous(), packed[-8:], scales[-8:], b, K))
    dy.zero_()
    dy[-1] = torch.arange(N, device="cuda") % 241 - 120
    for dt in (torch.bfloat16, torch.float32):
        dW = mpw.qlinear_grad_w_int8(dy, xq2, sx2, K, dtype=dt)
        assert torch.equal(dW, mpw.qlinear_grad_w_int8(dy[-1:], xq2[-1:], sx2[-1:], K, dtype=dt))
    assert mpw.device_error() == 0


# ---- gradients --------------------------------------------------------------


def _check_grad_x(mpw, M, N, K, b, layout):
    torch = _torch()
    W = _w(N, K, N + K + b)
    packed, scales = _rows(mpw, W, b, layout)
    dy = _dy(M, N, M)
    buf, dx = _guarded((M, K), torch.bfloat16, 7.0)
    mpw.qlinear_grad_x(dy.cuda(), packed, scales, b, K, dx=dx, layout=layout)
    q, s = oracle.quantize(W, b)
    ref, bound = oracle.grad_x_ref(dy.float().numpy(), q, s)
    _inside(dx, ref, bound, f"dx b={b} {layout} M={M} N={N} K={K}")
    assert _intact(buf, dx.numel(), 7.0)
    # independent roundings of at most 2^-8 of each factor and of the result
    if M * K >= 1000:
        err = np.linalg.norm(dx.double().cpu().numpy() - ref)
        assert err <= 2.0 ** -7.5 * np.linalg.norm(ref)


GRADS = [(1, 1, 1), (2, 3, 5), (16, 64, 128), (40, 100, 96), (130, 257, 333), (64, 1024, 512), (515, 1031, 777),
         (300, 130, 1280), (3, 1000, 2056)]


@pytest.mark.parametrize("M,N,K", GRADS)
@pytest.mark.parametrize("b", [4, 6, 8])
def test_grad_x(mpw, M, N, K, b):
    _check_grad_x(mpw, M, N, K, b, "canonical")


@pytest.mark.parametrize("M", [50, 700])
@pytest.mark.parametrize("layout", ["canonical", "paired"])
@pytest.mark.parametrize("b", list(range(4, 16)))
def test_grad_x_every_width(mpw, b, layout, M):
    _check_grad_x(mpw, M, 200, 288, b, layout)


@pytest.mark.parametrize("M", [1, 2, 7, 16, 32, 33, 64, 65, 100, 128, 129, 200, 256, 257, 400, 512, 513, 1100])
def test_grad_x_every_token_count(mpw, M):
    _check_grad_x(mpw, M, 1300, 520, 6, "canonical")


@pytest.mark.parametrize("M", [3, 40, 150, 600])
@pytest.mark.parametrize("b", [4, 7, 8])
def test_grad_x_many_rows(mpw, M, b):
    _check_grad_x(mpw, M, 17408, 72, b, "canonical")


def _check_grad_w(mpw, M, N, K, fp32, accumulate=False):
    torch = _torch()
    x = _x(M, K, M + 1)
    dy = _dy(M, N, M + 2)
    xq, sx = mpw.quantize_x_int8(x.cuda())
    dt = torch.float32 if fp32 else torch.bfloat16
    buf, dW = _guarded((N, K), dt, 7.0)
    mpw.qlinear_grad_w_int8(dy.cuda(), xq, sx, K, dW=dW, accumulate=accumulate)
    codes, sxr = oracle.quantize_x_int8(x.float().numpy())
    ref, bound = oracle.grad_w_ref(dy.float().numpy(), codes, sxr, fp32)
    if accumulate:
        ref, bound = ref + 7.0, bound + 2 * (7.0 + np.abs(ref)) * 2.0 ** -23
    _inside(dW, ref, bound, f"dW fp32={fp32} M={M} N={N} K={K}")
    assert _intact(buf, dW.numel(), 7.0)
    if not accumulate and N * K >= 1000:
        err = np.linalg.norm(dW.double().cpu().numpy() - ref)
        assert err <= (2.0 ** -16 if fp32 else 2.0 ** -7.5) * np.linalg.norm(ref)


@pytest.mark.parametrize("M,N,K", GRADS)
@pytest.mark.parametrize("fp32", [False, True])
def test_grad_w(mpw, M, N, K, fp32):
    _check_grad_w(mpw, M, N, K, fp32)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("M,N,K", [(4100, 300, 500), (8200, 40, 72), (1, 300, 17408)])
def test_grad_w_many_tokens_and_one(mpw, M, N, K, fp32):
    _check_grad_w(mpw, M, N, K, fp32)


@pytest.mark.parametrize("M,N,K", [(16, 64, 128), (130, 257, 333), (300, 130, 1280), (4100, 300, 500)])
def test_grad_w_accumulates(mpw, M, N, K):
    _check_grad_w(mpw, M, N, K, True, accumulate=True)


@pytest.mark.parametrize("M", [20, 800])
def test_grad_x_rows_past_32_bits(mpw, M):
    """4.8 G codes (9.7 GB of them expanded): of dy only the last column is not zero."""
    torch = _torch()
    rows, times, K, b = 4096, 72, 16384, 4
    block, scales = mpw.quantize_pack(workloads.gen_weight_torch(rows, K, 0.02, 5), b)
    dy = torch.zeros((M, rows * times), dtype=torch.bfloat16, device="cuda")
    dy[:, -1] = _dy(M, 1, 3).cuda()[:, 0]
    dx = mpw.qlinear_grad_x(dy, block.repeat(times, 1), scales.repeat(times), b, K)
    assert torch.equal(dx, mpw.qlinear_grad_x(dy[:, -8:].contiguous(), block[-8:], scales[-8:], b, K))
    assert mpw.device_error() == 0


@pytest.mark.parametrize("fp32", [False, True])
def test_grad_w_results_past_32_bits(mpw, fp32):
    """4.8 G results, a block of rows again and again; one token: sums of one product."""
    torch = _torch()
    rows, times, K = 4096, 72, 16384
    dt = torch.float32 if fp32 else torch.bfloat16
    xq, sx = mpw.quantize_x_int8(workloads.gen_x(1, K, 4).cuda())
    dy = _dy(1, rows, 5).cuda()
    ref = mpw.qlinear_grad_w_int8(dy, xq, sx, K, dtype=dt)
    dW = mpw.qlinear_grad_w_int8(dy.repeat(1, times), xq, sx, K, dtype=dt)
    for t in range(times):
        assert torch.equal(dW[t * rows:(t + 1) * rows], ref)
    assert mpw.device_error() == 0


def test_gradients_are_the_differences_of_the_product(mpw):
    """<dx, d> and <dW, e> against differences of L = sum dy * y in fp64."""
    torch = _torch()
    M, N, K, b = 37, 90, 160, 5
    W, x, dy = _w(N, K, 1), _x(M, K, 2), _dy(M, N, 3)
    packed, scales = _rows(mpw, W, b, "canonical")
    xq, sx = mpw.quantize_x_int8(x.cuda())
    dx = mpw.qlinear_grad_x(dy.cuda(), packed, scales, b, K).double().cpu().numpy()
    dW = mpw.qlinear_grad_w_int8(dy.cuda(), xq, sx, K, dtype=torch.float32).double().cpu().numpy()
    xh = mpw.dequantize(xq, sx, K, 8).double().cpu().numpy()
    wh = mpw.dequantize(packed, scales, K, b).double().cpu().numpy()
    dyf = dy.double().numpy()
    rng = np.random.default_rng(4)
    d, e = rng.standard_normal((M, K)), rng.standard_normal((N, K))
    h = 2.0 ** -6

    def loss(a, w):
        return float(np.sum(dyf * (a @ w.T)))

    want_x = (loss(xh + h * d, wh) - loss(xh - h * d, wh)) / (2 * h)
    want_w = (loss(xh, wh + h * e) - loss(xh, wh - h * e)) / (2 * h)
    lim_x = np.sum(np.abs(d) * oracle.grad_x_ref(dyf, *oracle.quantize(W, b))[1])
    lim_w = np.sum(np.abs(e) * oracle.grad_w_ref(dyf, *oracle.quantize_x_int8(x.float().numpy()), True)[1])
    assert abs(np.sum(dx * d) - want_x) <= lim_x + 1e-9
    assert abs(np.sum(dW * e) - want_w) <= lim_w + 1e-9


def test_non_finite_gradients_stay_in_their_rows(mpw):
    torch = _torch()
    M, N, K = 20, 64, 96
    packed, scales = _rows(mpw, _w(N, K, 1), 6, "canonical")
    dy = _dy(M, N, 3).cuda()
    want = mpw.qlinear_grad_x(dy, packed, scales, 6, K)
    dy[7, 5] = float("nan")
    dx = mpw.qlinear_grad_x(dy, packed, scales, 6, K)
    assert torch.isnan(dx[7]).all()
    keep = [i for i in range(M) if i != 7]
    assert torch.equal(dx[keep], want[keep])
    xq, sx = mpw.quantize_x_int8(_x(M, K, 4).cuda())
    dW = mpw.qlinear_grad_w_int8(dy, xq, sx, K)
    assert torch.isnan(dW[5]).any() and torch.isfinite(dW[[n for n in range(N) if n != 5]]).all()


# ---- together ---------------------------------------------------------------


def test_two_layer_step_and_sensitivities(mpw):
    """A step through two packed linears from 8-bit checkpoints, its gradients
    against fp64, and the accumulated weight gradients to the allocator."""
    torch = _torch()
    M, D, H = 48, 256, 640
    W1, W2 = _w(H, D, 1), _w(D, H, 2)
    p1, s1 = _rows(mpw, W1, 6, "canonical")
    p2, s2 = _rows(mpw, W2, 5, "canonical")
    g1 = torch.zeros((H, D), device="cuda")
    g2 = torch.zeros((D, H), device="cuda")
    r1, r2, l1, l2 = 0.0, 0.0, 0.0, 0.0
    q1, q2 = oracle.quantize(W1, 6), oracle.quantize(W2, 5)
    for step in range(3):
        x, dy = _x(M, D, 10 + step).cuda(), _dy(M, D, 20 + step).cuda()
        xq, sx = mpw.quantize_x_int8(x)
        h = mpw.qlinear_int8(x, p1, s1, 6, xq=xq, sx=sx)
        hq, sh = mpw.quantize_x_int8(h)
        y = mpw.qlinear_int8(h, p2, s2, 5, xq=hq, sx=sh)
        dh = mpw.qlinear_grad_x(dy, p2, s2, 5, H)
        mpw.qlinear_grad_w_int8(dy, hq, sh, H, dW=g2, accumulate=True)
        mpw.qlinear_grad_w_int8(dh, xq, sx, D, dW=g1, accumulate=True)
        # each link from the GPU's own input of that link
        hc = oracle.quantize_x_int8(h.float().cpu().numpy())
        xc = oracle.quantize_x_int8(x.float().cpu().numpy())
        _inside(y, *oracle.qlinear_int8_ref(*hc, *q2), "y")
        _inside(dh, *oracle.grad_x_ref(dy.float().cpu().numpy(), *q2), "dh")
        a, b = oracle.grad_w_ref(dy.float().cpu().numpy(), *hc, True)
        r2, l2 = r2 + a, l2 + b + 4 * (np.abs(r2) + np.abs(a)) * 2.0 ** -23
        a, b = oracle.grad_w_ref(dh.float().cpu().numpy(), *xc, True)
        r1, l1 = r1 + a, l1 + b + 4 * (np.abs(r1) + np.abs(a)) * 2.0 ** -23
    _inside(g1, r1, l1, "dW1")
    _inside(g2, r2, l2, "dW2")
    sens = [float(g.double().square().sum()) * float(np.mean(W.astype(np.float64) ** 2)) for g, W in ((g1, W1), (g2, W2))]
    shapes = [(H, D), (D, H)]
    floor = sum(n * mpw.packed_row_bytes(k, 4) + 4 * n for n, k in shapes)
    bits, total = mpw.allocate_bits(sens, shapes, floor * 2)
    assert all(4 <= v <= 16 for v in bits) and total <= floor * 2


def _all_ops(mpw, x, dy, packed, scales, b, K):
    torch = _torch()
    xq, sx = mpw.quantize_x_int8(x)
    y = mpw.qlinear_int8(None, packed, scales, b, xq=xq, sx=sx, K=K)
    dx = mpw.qlinear_grad_x(dy, packed, scales, b, K)
    dW = mpw.qlinear_grad_w_int8(dy, xq, sx, K, dtype=torch.float32)
    return y, dx, dW


@pytest.mark.parametrize("M", [1, 24, 300, 1100])
def test_captured_graphs_replay_with_new_inputs(mpw, M):
    """Two graphs captured one after another, replayed in turn: neither
    touches the other's scratch."""
    torch = _torch()
    N, K, b = 515, 320, 5
    packed, scales = _rows(mpw, _w(N, K, 1), b, "canonical")
    xs = [_x(M, K, i).cuda() for i in range(4)]
    dys = [_dy(M, N, i).cuda() for i in range(4)]
    want = [_all_ops(mpw, x, dy, packed, scales, b, K) for x, dy in zip(xs, dys)]
    graphs = []
    for i in range(2):
        x, dy = xs[i].clone(), dys[i].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _all_ops(mpw, x, dy, packed, scales, b, K)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _all_ops(mpw, x, dy, packed, scales, b, K)
        graphs.append((g, x, dy, out))
    for turn in range(4):
        for j, (g, x, dy, out) in enumerate(graphs):
            k = (turn + j) % 4
            x.copy_(xs[k])
            dy.copy_(dys[k])
            g.replay()
            for a, r in zip(out, want[k]):
                assert torch.equal(a, r)
    assert mpw.device_error() == 0


@pytest.mark.parametrize("M", [2, 40, 300, 1100])
def test_two_streams_at_once(mpw, M):
    torch = _torch()
    N, K, b = 1000, 1024, 6
    packed, scales = _rows(mpw, _w(N, K, 1), b, "canonical")
    xs = [_x(M, K, i).cuda() for i in range(2)]
    dys = [_dy(M, N, i).cuda() for i in range(2)]
    want = [_all_ops(mpw, x, dy, packed, scales, b, K) for x, dy in zip(xs, dys)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(_all_ops(mpw, xs[i], dys[i], packed, scales, b, K))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            for a, r in zip(out, want[i]):
                assert torch.equal(a, r)


@pytest.mark.parametrize("M", [1, 40, 300, 900])
def test_rows_quantized_by_the_call_before(mpw, M):
    """Quantized activations are packed rows: a product that follows them at once reads the new ones."""
    torch = _torch()
    N, K = 20000, 2048
    xq, sx = mpw.quantize_x_int8(workloads.gen_x(M, K, 1).cuda())
    dy = _dy(M, N, 2).cuda()
    keys = [workloads.gen_x(N, K, 3 + i).cuda() for i in range(3)]
    rows = torch.empty((N, K), dtype=torch.uint8, device="cuda")
    scales = torch.empty((N,), dtype=torch.float32, device="cuda")

    def both(wait):
        out = []
        for op in (lambda: mpw.qlinear_int8(None, rows, scales, 8, xq=xq, sx=sx, K=K),
                   lambda: mpw.qlinear_grad_x(dy, rows, scales, 8, K)):
            for key in keys:
                mpw.quantize_x_int8(key, xq=rows, sx=scales)
                if wait:
                    torch.cuda.synchronize()
                out.append(op())
        return out

    for _ in range(3):
        for got, want in zip(both(False), both(True)):
            assert torch.equal(got, want)


def test_stream_argument_and_callers_workspace(mpw):
    torch = _torch()
    M, N, K, b = 1050, 264, 512, 7
    packed, scales = _rows(mpw, _w(N, K, 1), b, "canonical")
    x, dy = _x(M, K, 0).cuda(), _dy(M, N, 0).cuda()
    y0, dx0, dW0 = _all_ops(mpw, x, dy, packed, scales, b, K)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    xq, sx = mpw.quantize_x_int8(x, stream=st)
    y = mpw.qlinear_int8(None, packed, scales, b, xq=xq, sx=sx, K=K, stream=st)
    dx = mpw.qlinear_grad_x(dy, packed, scales, b, K, stream=st)
    dW = mpw.qlinear_grad_w_int8(dy, xq, sx, K, dtype=torch.float32, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(dx, dx0) and torch.equal(dW, dW0)
    # a dirty workspace of the smallest size that is asked for
    L = mpw.lib
    n = max(L.mpw_qlinear_int8_workspace_bytes(b, 0, M, N, K), L.mpw_qlinear_grad_x_workspace_bytes(b, 0, M, N, K),
            L.mpw_qlinear_grad_w_int8_workspace_bytes(mpw.GRAD_F32, M, N, K))
    buf, ws = _guarded((n,), torch.uint8, 0xEE)
    y = mpw.qlinear_int8(None, packed, scales, b, xq=xq, sx=sx, K=K, workspace=ws)
    dx = mpw.qlinear_grad_x(dy, packed, scales, b, K, workspace=ws)
    dW = mpw.qlinear_grad_w_int8(dy, xq, sx, K, dtype=torch.float32, workspace=ws)
    assert torch.equal(y, y0) and torch.equal(dx, dx0) and torch.equal(dW, dW0)
    assert _intact(buf, n, 0xEE)


def test_temporaries_of_another_stream_are_not_handed_out(mpw):
    """Everything a call allocates for a busy side stream stays its own while
    the current stream allocates and writes the same sizes."""
    torch = _torch()
    M, N, K, b = 1100, 264, 512, 6
    packed, scales = _rows(mpw, _w(N, K, 1), b, "canonical")
    x, dy = _x(M, K, 0).cuda(), _dy(M, N, 0).cuda()
    want = _all_ops(mpw, x, dy, packed, scales, b, K)
    sizes = [(M, mpw.packed_row_bytes(K, 8)), (4 * M,), (N * K,), (6 * M * K,), (2 * M * N,), (4 * N * K,)]
    st = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            torch.cuda._sleep(20_000_000)
        y = mpw.qlinear_int8(x, packed, scales, b, stream=st)
        dx = mpw.qlinear_grad_x(dy, packed, scales, b, K, stream=st)
        xq, sx = mpw.quantize_x_int8(x, stream=st)
        dW = mpw.qlinear_grad_w_int8(dy, xq, sx, K, dtype=torch.float32, stream=st)
        for n in sizes:
            for _ in range(3):
                torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x55)
        st.synchronize()
        for a, r in zip((y, dx, dW), want):
            assert torch.equal(a, r)


def test_refusals(mpw):
    torch = _torch()
    M, N, K = 40, 24, 64
    packed, scales = _rows(mpw, _w(N, K, 1), 6, "canonical")
    x, dy = _x(M, K, 0).cuda(), _dy(M, N, 0).cuda()
    xq, sx = mpw.quantize_x_int8(x)
    with pytest.raises(ValueError):
        mpw.quantize_x_int8(x.t())
    with pytest.raises(ValueError):
        mpw.quantize_x_int8(x, xq=torch.empty((M, K + 16), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        mpw.qlinear_int8(None, packed, scales, 6, xq=xq, sx=sx[1:], K=K)
    with pytest.raises(ValueError):
        mpw.qlinear_int8(None, packed, scales, 6, xq=xq, sx=sx, K=K + 1)
    with pytest.raises(ValueError):
        mpw.qlinear_int8(x, packed, scales, 6, y=torch.empty((M, N + 1), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        mpw.qlinear_int8(x, packed, scales[1:], 6)
    with pytest.raises(ValueError):
        mpw.qlinear_grad_x(dy, packed[1:], scales[1:], 6, K)
    with pytest.raises(TypeError):
        mpw.qlinear_grad_x(dy.float(), packed, scales, 6, K)
    with pytest.raises(ValueError):
        mpw.qlinear_grad_w_int8(dy[1:], xq, sx, K)
    with pytest.raises(ValueError):
        mpw.qlinear_grad_w_int8(dy, xq, sx, K, accumulate=True)
    with pytest.raises(ValueError):
        mpw.qlinear_grad_w_int8(dy, xq, sx, K, dW=torch.empty((N, K), dtype=torch.bfloat16, device="cuda"),
                                accumulate=True)
    with pytest.raises(TypeError):
        mpw.qlinear_grad_w_int8(dy, xq, sx, K, dtype=torch.float16)
    with pytest.raises(ValueError):
        mpw.qlinear_grad_w_int8(dy, xq, sx, K, workspace=torch.empty((16,), dtype=torch.uint8, device="cuda"))
    p9, s9 = mpw.quantize_pack(torch.randn(N, K, device="cuda"), 9)
    with pytest.raises(mpw.MPWError) as e:
        mpw.qlinear_int8(x, p9, s9, 9)
    assert e.value.status == mpw.MPW_E_UNSUPPORTED_BITS
