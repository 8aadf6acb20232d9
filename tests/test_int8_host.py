"""Host-side checks of the int8 linear's and the gradients' entry points: bad
arguments are refused before anything is launched, workspace sizes, and the
binding's own checks.  No call here reaches a CUDA kernel."""
import pytest
import torch

import mixed_precision_weight_row_b200 as mpw

A, B, C, D, E, W = (0x10000 * i for i in range(1, 7))    # fake 16-byte aligned addresses
BIG = 1 << 40

INV, BITS, ALIGN = mpw.MPW_E_INVALID_ARG, mpw.MPW_E_UNSUPPORTED_BITS, mpw.MPW_E_MISALIGNED


def test_quantize_x_int8_validation():
    f = mpw.lib.mpw_quantize_x_int8
    for args in [(0, 4, 16, B, C), (A, 4, 16, 0, C), (A, 4, 16, B, 0), (A, 0, 16, B, C), (A, 4, 0, B, C),
                 (A, -1, 16, B, C), (A, 4, -3, B, C), (A, 1 << 31, 16, B, C), (A, 4, 1 << 31, B, C)]:
        assert f(*args, 0) == INV, args
    for args in [(A + 1, 4, 16, B, C), (A, 4, 16, B + 8, C), (A, 4, 16, B, C + 2)]:
        assert f(*args, 0) == ALIGN, args


def _lin(xq=A, sx=B, packed=C, scales=D, bits=6, layout=0, M=64, N=32, K=64, y=E, ws=W, nb=BIG):
    return mpw.lib.mpw_qlinear_int8(xq, sx, packed, scales, bits, layout, M, N, K, y, ws, nb, 0)


def test_qlinear_int8_validation():
    for b in (3, 9, 12, 16):
        assert _lin(bits=b) == BITS
    for kw in [dict(xq=0), dict(sx=0), dict(packed=0), dict(scales=0), dict(y=0), dict(M=0), dict(N=0), dict(K=0),
               dict(M=-1), dict(layout=2), dict(layout=-1), dict(K=131072), dict(layout=1, K=48), dict(N=1 << 31)]:
        assert _lin(**kw) == INV, kw
    for kw in [dict(xq=A + 8), dict(sx=B + 2), dict(packed=C + 4), dict(scales=D + 1), dict(y=E + 1)]:
        assert _lin(**kw) == ALIGN, kw


def _gx(dy=A, packed=B, scales=C, bits=6, layout=0, M=64, N=32, K=64, dx=D, ws=W, nb=BIG):
    return mpw.lib.mpw_qlinear_grad_x(dy, packed, scales, bits, layout, M, N, K, dx, ws, nb, 0)


def test_grad_x_validation():
    for b in (3, 16):
        assert _gx(bits=b) == BITS
    for kw in [dict(dy=0), dict(packed=0), dict(scales=0), dict(dx=0), dict(M=0), dict(N=0), dict(K=0), dict(layout=3),
               dict(layout=1, K=48), dict(M=1 << 30), dict(ws=0, M=4000),
               dict(M=4000, nb=mpw.lib.mpw_qlinear_grad_x_workspace_bytes(6, 0, 4000, 32, 64) - 1)]:
        assert _gx(**kw) == INV, kw
    for kw in [dict(dy=A + 2), dict(dy=A + 1, N=33), dict(packed=B + 8), dict(scales=C + 2), dict(dx=D + 1),
               dict(ws=W + 8, M=4000)]:
        assert _gx(**kw) == ALIGN, kw


def _gw(dy=A, xq=B, sx=C, M=64, N=32, K=64, dW=D, kind=0, acc=0, ws=W, nb=BIG):
    return mpw.lib.mpw_qlinear_grad_w_int8(dy, xq, sx, M, N, K, dW, kind, acc, ws, nb, 0)


def test_grad_w_validation():
    for kw in [dict(dy=0), dict(xq=0), dict(sx=0), dict(dW=0), dict(M=0), dict(N=-2), dict(K=0), dict(kind=2),
               dict(kind=-1), dict(acc=1), dict(ws=0),
               dict(nb=mpw.lib.mpw_qlinear_grad_w_int8_workspace_bytes(0, 64, 32, 64) - 1)]:
        assert _gw(**kw) == INV, kw
    for kw in [dict(dy=A + 2), dict(dy=A + 1, N=33), dict(xq=B + 4), dict(sx=C + 2), dict(dW=D + 1),
               dict(kind=1, dW=D + 2), dict(ws=W + 4)]:
        assert _gw(**kw) == ALIGN, kw


def test_workspace_sizes_of_bad_arguments_are_zero():
    L = mpw.lib
    for args in [(3, 0, 4, 4, 4), (9, 0, 4, 4, 4), (6, 2, 4, 4, 4), (6, 0, 0, 4, 4), (6, 0, 4, 4, 131072)]:
        assert L.mpw_qlinear_int8_workspace_bytes(*args) == 0
    for args in [(3, 0, 4, 4, 4), (16, 0, 4, 4, 4), (6, -1, 4, 4, 4), (6, 0, 4, 0, 4)]:
        assert L.mpw_qlinear_grad_x_workspace_bytes(*args) == 0
    for args in [(2, 4, 4, 4), (0, 0, 4, 4), (1, 4, 4, 0)]:
        assert L.mpw_qlinear_grad_w_int8_workspace_bytes(*args) == 0


def test_binding_refuses_what_is_no_cuda_tensor():
    x = torch.zeros((4, 16), dtype=torch.bfloat16)
    rows = torch.zeros((4, 16), dtype=torch.uint8)
    s = torch.ones(4)
    with pytest.raises(ValueError):
        mpw.quantize_x_int8(x)
    with pytest.raises(TypeError):
        mpw.quantize_x_int8(x.float())
    with pytest.raises(ValueError):
        mpw.qlinear_int8(None, rows, s, 8, xq=rows)          # xq without sx
    with pytest.raises(ValueError):
        mpw.qlinear_int8(None, rows, s, 8, xq=rows, sx=s)    # no K
    with pytest.raises(ValueError):
        mpw.qlinear_grad_x(x, rows, s, 8, 16)
    with pytest.raises(ValueError):
        mpw.qlinear_grad_w_int8(x, rows, s, 16)


def test_binding_refuses_incomplete_activations_before_anything_else():
    x = torch.zeros((4, 16), dtype=torch.bfloat16)
    rows = torch.zeros((4, 16), dtype=torch.uint8)
    s = torch.ones(4)
    for kw in (dict(xq=rows), dict(sx=s)):
        with pytest.raises(ValueError, match="xq and sx"):
            mpw.qlinear_int8(x, rows, s, 8, **kw)
    with pytest.raises(ValueError, match="K is needed"):
        mpw.qlinear_int8(None, rows, s, 8, xq=rows, sx=s)


def test_overlapping_outputs_are_refused():
    """An output, or the workspace, that shares bytes with an input or with one
    another: blocks that finish early would overwrite what others still read."""
    f = mpw.lib.mpw_quantize_x_int8                       # x 64 x 64 bf16: 8192 bytes, xq 4096, sx 256
    for args in [(A, 64, 64, A, C), (A, 64, 64, A + 8176, C), (A + 4080, 64, 64, A, C), (A, 64, 64, B, A + 8188),
                 (A, 64, 64, B, B + 4092), (A, 64, 64, B, B - 252)]:
        assert f(*args, 0) == INV, args
    # xq 64 x 64: 4096 bytes, sx 256, packed 32 x 48: 1536, scales 128, y 64 x 32 bf16: 4096
    for kw in [dict(y=A), dict(y=A + 4094), dict(y=A - 4094), dict(y=B + 254), dict(y=C), dict(y=C + 1534), dict(y=D),
               dict(y=D - 4094)]:
        assert _lin(**kw) == INV, kw
    need = mpw.lib.mpw_qlinear_int8_workspace_bytes(6, 0, 9000, 512, 64)
    assert need == 512 * 64
    big = dict(M=9000, N=512, xq=1 << 24, y=1 << 26, nb=need)
    for kw in [dict(ws=C), dict(ws=1 << 24), dict(ws=(1 << 26) + 16), dict(ws=(1 << 26) - need + 16), dict(ws=D),
               dict(ws=B)]:
        assert _lin(**{**big, **kw}) == INV, kw
    # dy 64 x 64 bf16: 8192 bytes, packed 64 x 48, scales 256, dx 64 x 64 bf16
    for kw in [dict(dx=A), dict(dx=A + 8190), dict(dx=B + 3070), dict(dx=C), dict(dx=C - 8190)]:
        assert _gx(**{**dict(N=64), **kw}) == INV, kw
    # dy 64 x 32 bf16: 4096 bytes, xq 4096, sx 256, dW 32 x 64
    for kw in [dict(dW=A + 4094), dict(dW=B), dict(dW=C + 254), dict(kind=1, dW=A - 8188), dict(dW=W), dict(ws=A),
               dict(ws=B - 16), dict(ws=C)]:
        assert _gw(**kw) == INV, kw
