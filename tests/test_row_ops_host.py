"""Refusals and sizes of the row operators, on the CPU: every invalid call
returns its status before any device work, and the torch wrappers raise."""
import pytest
import torch

import convolution_implicit_gemm_fwd_amd as cim
from convolution_implicit_gemm_fwd_amd import abi

A, B, C, D, E, F, G = (k << 32 for k in range(1, 8))     # addresses far apart, never touched
BF16, FP32, FP16, MX = 0, 1, 2, 3


def ln(**kw):
    a = dict(x=A, ldx=64, gamma=B, beta=C, rows=8, cols=64, eps=1e-5, x_dtype=BF16, y_dtype=FP32, y=D, mean=E, rstd=F,
             stream=0)
    a.update(kw)
    return abi.layer_norm_fwd(**a)


def lnq(**kw):
    a = dict(x=A, ldx=64, gamma=B, beta=C, rows=8, cols=64, eps=1e-5, x_dtype=BF16, codes=D, scales=E, mean=None,
             rstd=None, stream=0)
    a.update(kw)
    return abi.layer_norm_fwd_mxfp4(**a)


def lnb(**kw):
    a = dict(dy=A, lddy=64, x=B, ldx=64, gamma=C, mean=D, rstd=D + 4096, rows=8, cols=64, dy_dtype=BF16, x_dtype=BF16,
             dx_dtype=BF16, dx=E, dgamma=F, dbeta=F + 4096, ws=G, ws_bytes=1 << 20, stream=0)
    a.update(kw)
    return abi.layer_norm_bwd(**a)


def quant(**kw):
    a = dict(x=A, ldx=64, rows=8, cols=64, dtype=BF16, transpose=0, codes=B, scales=C, stream=0)
    a.update(kw)
    return abi.mxfp4_quantize(**a)


def deq(**kw):
    a = dict(codes=A, scales=B, rows=8, cols=64, dtype=BF16, out=C, stream=0)
    a.update(kw)
    return abi.mxfp4_dequantize(**a)


def lin(**kw):
    a = dict(x=A, ldx=64, x_scales=None, x_dtype=BF16, w_codes=B, w_scales=C, bias=D, M=8, N=48, K=64, out_dtype=FP32,
             out=E, ws=F, ws_bytes=1 << 20, stream=0)
    a.update(kw)
    return abi.mxfp4_linear_fwd(**a)


def linb(**kw):
    a = dict(dy=A, lddy=48, dy_dtype=BF16, x=B, ldx=64, w=C, ldw=64, dtype=BF16, M=8, N=48, K=64, dx_dtype=BF16, dx=D,
             dw=E, db=F, ws=G, ws_bytes=1 << 20, stream=0)
    a.update(kw)
    return abi.mxfp4_linear_bwd(**a)


CASES = [
    (ln, abi.CONVIMG_ERR_SHAPE, [dict(rows=-1), dict(cols=0), dict(cols=-3), dict(ldx=63)]),
    (ln, abi.CONVIMG_ERR_DTYPE, [dict(x_dtype=MX), dict(y_dtype=3), dict(x_dtype=-1)]),
    (ln, abi.CONVIMG_ERR_RANGE, [dict(rows=1 << 31)]),
    (ln, abi.CONVIMG_ERR_NULL, [dict(x=None), dict(y=None)]),
    (ln, abi.CONVIMG_ERR_ALIAS, [dict(y=A), dict(y=A + 1022), dict(mean=A + 8), dict(rstd=C), dict(rstd=E + 28),
                                 dict(mean=D + 4)]),
    (lnq, abi.CONVIMG_ERR_NULL, [dict(x=None), dict(codes=None), dict(scales=None)]),
    (lnq, abi.CONVIMG_ERR_ALIGN, [dict(codes=D + 8), dict(scales=E + 2)]),
    (lnq, abi.CONVIMG_ERR_ALIAS, [dict(codes=A), dict(scales=D + 252), dict(scales=B)]),
    (lnb, abi.CONVIMG_ERR_SHAPE, [dict(rows=-1), dict(cols=0), dict(lddy=63), dict(ldx=1)]),
    (lnb, abi.CONVIMG_ERR_DTYPE, [dict(dy_dtype=4), dict(x_dtype=3), dict(dx_dtype=3)]),
    (lnb, abi.CONVIMG_ERR_NULL, [dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=None),
                                 dict(dgamma=None), dict(dbeta=None), dict(ws=None)]),
    (lnb, abi.CONVIMG_ERR_WORKSPACE, [dict(ws_bytes=0), dict(ws_bytes=63)]),
    (lnb, abi.CONVIMG_ERR_ALIGN, [dict(ws=G + 4)]),
    (lnb, abi.CONVIMG_ERR_ALIAS, [dict(dx=A), dict(dx=B + 2), dict(dgamma=C), dict(dbeta=F + 4), dict(ws=E)]),
    (quant, abi.CONVIMG_ERR_SHAPE, [dict(rows=-1), dict(cols=0), dict(ldx=63), dict(rows=0, transpose=1)]),
    (quant, abi.CONVIMG_ERR_DTYPE, [dict(dtype=MX)]),
    (quant, abi.CONVIMG_ERR_RANGE, [dict(rows=1 << 20, cols=1 << 12, ldx=1 << 12)]),
    (quant, abi.CONVIMG_ERR_NULL, [dict(x=None), dict(codes=None), dict(scales=None)]),
    (quant, abi.CONVIMG_ERR_ALIGN, [dict(codes=B + 4), dict(scales=C + 1)]),
    (quant, abi.CONVIMG_ERR_ALIAS, [dict(codes=A + 16), dict(scales=A), dict(scales=B + 252)]),
    (deq, abi.CONVIMG_ERR_SHAPE, [dict(rows=-1), dict(cols=0)]),
    (deq, abi.CONVIMG_ERR_DTYPE, [dict(dtype=MX)]),
    (deq, abi.CONVIMG_ERR_NULL, [dict(codes=None), dict(scales=None), dict(out=None)]),
    (deq, abi.CONVIMG_ERR_ALIGN, [dict(codes=A + 8), dict(scales=B + 2)]),
    (deq, abi.CONVIMG_ERR_ALIAS, [dict(out=A), dict(out=B + 4)]),
    (lin, abi.CONVIMG_ERR_SHAPE, [dict(M=-1), dict(N=0), dict(K=0), dict(ldx=63)]),
    (lin, abi.CONVIMG_ERR_DTYPE, [dict(x_dtype=4), dict(out_dtype=MX)]),
    (lin, abi.CONVIMG_ERR_RANGE, [dict(N=1 << 20, K=1 << 12, ldx=1 << 12)]),
    (lin, abi.CONVIMG_ERR_NULL, [dict(x=None), dict(w_codes=None), dict(w_scales=None), dict(out=None), dict(ws=None),
                                 dict(x_dtype=MX)]),
    (lin, abi.CONVIMG_ERR_ALIGN, [dict(w_codes=B + 8), dict(w_scales=C + 2), dict(ws=F + 8),
                                  dict(x_dtype=MX, x=A + 4, x_scales=G)]),
    (lin, abi.CONVIMG_ERR_WORKSPACE, [dict(ws_bytes=16)]),
    (lin, abi.CONVIMG_ERR_ALIAS, [dict(out=A), dict(out=D), dict(ws=B), dict(ws=E), dict(out=C)]),
    (linb, abi.CONVIMG_ERR_SHAPE, [dict(M=-1), dict(N=0), dict(K=0), dict(lddy=47), dict(ldx=63), dict(ldw=63)]),
    (linb, abi.CONVIMG_ERR_DTYPE, [dict(dy_dtype=MX), dict(dtype=MX), dict(dx_dtype=3)]),
    (linb, abi.CONVIMG_ERR_NULL, [dict(dy=None), dict(x=None), dict(w=None), dict(dx=None), dict(dw=None),
                                  dict(ws=None)]),
    (linb, abi.CONVIMG_ERR_ALIGN, [dict(ws=G + 4)]),
    (linb, abi.CONVIMG_ERR_WORKSPACE, [dict(ws_bytes=256)]),
    (linb, abi.CONVIMG_ERR_ALIAS, [dict(dx=B), dict(dw=C), dict(db=A), dict(ws=E), dict(db=E + 64)]),
]


@pytest.mark.parametrize("fn,status,calls", CASES, ids=lambda v: getattr(v, "__name__", None) or "")
def test_refusals(fn, status, calls):
    for kw in calls:
        assert fn(**kw) == status, "%s(%s)" % (fn.__name__, kw)


def test_sizes():
    assert abi.mxfp4_bytes(5, 33) == (0, 5 * 2 * 16, 5 * 4)
    assert abi.mxfp4_bytes(0, 1) == (0, 0, 0)
    assert abi.mxfp4_bytes(7, 129) == (0, 7 * 5 * 16, 2 * 7 * 4)
    assert abi.mxfp4_bytes(3, 0)[0] == abi.CONVIMG_ERR_SHAPE
    assert abi.mxfp4_bytes(1 << 20, 1 << 12)[0] == abi.CONVIMG_ERR_RANGE
    assert abi.mxfp4_linear_workspace(8, 8, 64, MX) == (0, 0)
    assert abi.mxfp4_linear_workspace(8, 0, 64, MX)[0] == abi.CONVIMG_ERR_SHAPE
    assert abi.layer_norm_bwd_workspace(-1, 4)[0] == abi.CONVIMG_ERR_SHAPE
    assert abi.mxfp4_linear_bwd_workspace(4, 4, 0)[0] == abi.CONVIMG_ERR_SHAPE
    rc, n = abi.mxfp4_linear_workspace(8, 16, 64, FP16)
    assert rc == 0 and n >= 8 * 32 + 8 * 4


def test_empty_batches_need_no_data():
    assert ln(rows=0, x=None, y=None, mean=None, rstd=None) == 0
    assert quant(rows=0, x=None) == 0
    assert deq(rows=0, out=None) == 0
    assert lin(M=0, x=None, out=None) == 0


def test_wrappers_refuse_host_tensors():
    x = torch.zeros(4, 64)
    for call in (lambda: cim.layer_norm_nhwc(x), lambda: cim.layer_norm_mxfp4_nhwc(x),
                 lambda: cim.mxfp4_quantize_nhwc(x),
                 lambda: cim.layer_norm_bwd_nhwc(x, x, None, x[:, 0], x[:, 0]),
                 lambda: cim.mxfp4_linear_bwd_nhwc(x, x, x)):
        with pytest.raises(ValueError):
            call()
    q = cim.Mxfp4Tensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8), 4, 64)
    with pytest.raises(ValueError):
        cim.mxfp4_dequantize_nhwc(q, torch.float32)
    with pytest.raises(ValueError):
        cim.mxfp4_linear_nhwc(x, q)


def test_row_geometry():
    from convolution_implicit_gemm_fwd_amd.rows import _rows_of

    class View:      # a device tensor's geometry
        is_cuda = True

        def __init__(self, t):
            self.shape, self._s = t.shape, t.stride()

        def stride(self):
            return self._s

    big = torch.empty(2, 3, 4, 96)
    assert _rows_of(View(big), "x") == (24, 96, 96)
    assert _rows_of(View(big[..., :64]), "x") == (24, 64, 96)
    assert _rows_of(View(big[:, :, :1, :64]), "x") == (6, 64, 384)
    assert _rows_of(View(big[0, 0, 0]), "x") == (1, 96, 96)
    assert _rows_of(View(torch.empty(5, 1)), "x") == (5, 1, 1)
    assert _rows_of(View(torch.empty(0, 7)), "x") == (0, 7, 7)
    assert _rows_of(View(torch.empty(3, 0, 7)), "x")[:2] == (0, 7)
    for bad in (big.transpose(2, 3), big[:, :2], torch.empty(1, 8).expand(4, 8), torch.empty(4, 0), torch.empty(())):
        with pytest.raises(ValueError):
            _rows_of(View(bad), "x")
