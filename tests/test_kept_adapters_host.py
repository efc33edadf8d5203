"""Refusals and sizes of the passes on activations kept in 8 bits and of the low-rank adapters, on the CPU: every invalid
call returns its status before any device work, and the torch wrappers raise."""
import types

import pytest
import torch

import convolution_implicit_gemm_fwd_amd as cim
from convolution_implicit_gemm_fwd_amd import abi
from convolution_implicit_gemm_fwd_amd import rows as R
from test_row_wrappers_host import HOME, SIDE, Dev, Machine, dev, far, tensors

A, B, C, D, E, F, G, H, I, J, K, L, M, N = (k << 32 for k in range(1, 15))     # addresses far apart, never touched
BF16, FP32, FP16, MX, KEPT = 0, 1, 2, 3, 4
COLS = (1 << 31) - (1 << 14)


def quant(**kw):
    a = dict(x=A, ldx=64, rows=8, cols=64, dtype=BF16, codes=B, scales=C, stream=0)
    a.update(kw)
    return abi.mxint8_quantize(**a)


def deq(**kw):
    a = dict(codes=A, scales=B, rows=8, cols=64, dtype=BF16, out=C, stream=0)
    a.update(kw)
    return abi.mxint8_dequantize(**a)


def ln(**kw):
    a = dict(x=A, ldx=64, gamma=B, beta=C, rows=8, cols=64, eps=1e-5, x_dtype=BF16, y_dtype=FP32, y=D, codes=E, scales=F,
             rstd=G, stream=0)
    a.update(kw)
    return abi.layer_norm_fwd_mxint8(**a)


def lnb(**kw):
    a = dict(dy=A, lddy=64, codes=B, scales=C, gamma=D, rstd=E, rows=8, cols=64, dy_dtype=BF16, dx_dtype=BF16, dx=F,
             dgamma=G, dbeta=G + 4096, ws=H, ws_bytes=1 << 20, stream=0)
    a.update(kw)
    return abi.layer_norm_bwd_mxint8(**a)


def linb(**kw):
    a = dict(dy=A, lddy=48, dy_dtype=BF16, x_codes=B, x_scales=C, w=D, ldw=64, w_dtype=BF16, M=8, N=48, K=64, dx_dtype=BF16,
             dx=E, dw=F, db=G, ws=H, ws_bytes=1 << 20, stream=0)
    a.update(kw)
    return abi.mxfp4_linear_bwd_mxint8(**a)


def fwd(**kw):
    a = dict(x=A, ldx=64, x_dtype=BF16, w_codes=B, w_scales=C, bias=D, down=E, up=F, scale=G, ids=H, adapters=3, rank=4,
             a_dtype=BF16, M=8, N=48, K=64, out_dtype=FP32, out=I, h=J, x_codes=K, x_scales=L, ws=M, ws_bytes=1 << 20,
             stream=0)
    a.update(kw)
    return abi.mxfp4_linear_adapters_fwd(**a)


def bwd(**kw):
    a = dict(dy=A, lddy=48, dy_dtype=BF16, x=B, ldx=64, x_scales=None, x_dtype=BF16, wt_codes=C, wt_scales=D, down=E, up=F,
             scale=G, ids=H, adapters=3, rank=4, a_dtype=BF16, h=I, M=8, N=48, K=64, dx_dtype=BF16, dx=J, ddown=K, dup=L,
             ws=M, ws_bytes=1 << 24, stream=0)
    a.update(kw)
    return abi.mxfp4_linear_adapters_bwd(**a)


CASES = [
    (quant, abi.CONVIMG_ERR_SHAPE, [dict(rows=-1), dict(cols=0), dict(ldx=63)]),
    (quant, abi.CONVIMG_ERR_DTYPE, [dict(dtype=MX), dict(dtype=KEPT), dict(dtype=-1)]),
    (quant, abi.CONVIMG_ERR_RANGE, [dict(rows=1 << 31), dict(rows=1, cols=COLS + 1, ldx=COLS + 1)]),
    (quant, abi.CONVIMG_ERR_NULL, [dict(x=None), dict(codes=None), dict(scales=None)]),
    (quant, abi.CONVIMG_ERR_ALIGN, [dict(codes=B + 8), dict(scales=C + 2)]),
    (quant, abi.CONVIMG_ERR_ALIAS, [dict(codes=A), dict(scales=A + 1020), dict(scales=B + 508), dict(codes=A + 1008)]),
    (deq, abi.CONVIMG_ERR_SHAPE, [dict(rows=-1), dict(cols=0)]),
    (deq, abi.CONVIMG_ERR_DTYPE, [dict(dtype=KEPT)]),
    (deq, abi.CONVIMG_ERR_NULL, [dict(codes=None), dict(scales=None), dict(out=None)]),
    (deq, abi.CONVIMG_ERR_ALIGN, [dict(codes=A + 4), dict(scales=B + 1)]),
    (deq, abi.CONVIMG_ERR_ALIAS, [dict(out=A + 510), dict(out=B + 28)]),
    (ln, abi.CONVIMG_ERR_SHAPE, [dict(rows=-1), dict(cols=0), dict(ldx=63)]),
    (ln, abi.CONVIMG_ERR_DTYPE, [dict(x_dtype=MX), dict(y_dtype=KEPT)]),
    (ln, abi.CONVIMG_ERR_RANGE, [dict(rows=1 << 31)]),
    (ln, abi.CONVIMG_ERR_NULL, [dict(x=None), dict(y=None), dict(codes=None), dict(scales=None), dict(rstd=None)]),
    (ln, abi.CONVIMG_ERR_ALIGN, [dict(codes=E + 8), dict(scales=F + 2)]),
    (ln, abi.CONVIMG_ERR_ALIAS, [dict(y=A), dict(codes=A + 16), dict(scales=D), dict(rstd=E + 508), dict(rstd=B), dict(y=C)]),
    (lnb, abi.CONVIMG_ERR_SHAPE, [dict(rows=-1), dict(cols=0), dict(lddy=63)]),
    (lnb, abi.CONVIMG_ERR_DTYPE, [dict(dy_dtype=KEPT), dict(dx_dtype=MX)]),
    (lnb, abi.CONVIMG_ERR_NULL, [dict(dy=None), dict(codes=None), dict(scales=None), dict(rstd=None), dict(dx=None),
                                 dict(dgamma=None), dict(dbeta=None), dict(ws=None)]),
    (lnb, abi.CONVIMG_ERR_ALIGN, [dict(ws=H + 4), dict(codes=B + 8), dict(scales=C + 2)]),
    (lnb, abi.CONVIMG_ERR_WORKSPACE, [dict(ws_bytes=0)]),
    (lnb, abi.CONVIMG_ERR_ALIAS, [dict(dx=A), dict(dx=B), dict(dgamma=C), dict(dbeta=G + 4), dict(ws=F), dict(dx=E)]),
    (linb, abi.CONVIMG_ERR_SHAPE, [dict(M=-1), dict(N=0), dict(K=0), dict(lddy=47), dict(ldw=63)]),
    (linb, abi.CONVIMG_ERR_DTYPE, [dict(dy_dtype=MX), dict(w_dtype=KEPT), dict(dx_dtype=3)]),
    (linb, abi.CONVIMG_ERR_NULL, [dict(dy=None), dict(x_codes=None), dict(x_scales=None), dict(w=None), dict(dx=None),
                                  dict(dw=None), dict(ws=None)]),
    (linb, abi.CONVIMG_ERR_ALIGN, [dict(ws=H + 4), dict(x_codes=B + 8), dict(x_scales=C + 2)]),
    (linb, abi.CONVIMG_ERR_WORKSPACE, [dict(ws_bytes=256)]),
    (linb, abi.CONVIMG_ERR_ALIAS, [dict(dx=B), dict(dw=C), dict(db=A), dict(ws=E), dict(dw=B + 508), dict(dx=D)]),
    (fwd, abi.CONVIMG_ERR_SHAPE, [dict(M=-1), dict(N=0), dict(K=0), dict(ldx=63), dict(adapters=0), dict(rank=0),
                                  dict(adapters=-1), dict(rank=-4)]),
    (fwd, abi.CONVIMG_ERR_DTYPE, [dict(x_dtype=MX), dict(x_dtype=KEPT), dict(a_dtype=MX), dict(out_dtype=KEPT)]),
    (fwd, abi.CONVIMG_ERR_RANGE, [dict(rank=4097), dict(N=1 << 25), dict(M=1, K=1 << 25, ldx=1 << 25), dict(M=1 << 26),
                                  dict(N=1 << 20, K=1 << 12, ldx=1 << 12)]),
    (fwd, abi.CONVIMG_ERR_NULL, [dict([(n, None)]) for n in ("x", "w_codes", "w_scales", "down", "up", "scale", "ids", "out",
                                                             "x_codes", "x_scales", "ws")]),
    (fwd, abi.CONVIMG_ERR_ALIGN, [dict(w_codes=B + 8), dict(w_scales=C + 2), dict(ws=M + 8), dict(x_codes=K + 8),
                                  dict(x_scales=L + 2)]),
    (fwd, abi.CONVIMG_ERR_WORKSPACE, [dict(ws_bytes=16)]),
    (fwd, abi.CONVIMG_ERR_ALIAS, [dict(out=A), dict(out=E + 8), dict(h=F), dict(h=I), dict(x_codes=A), dict(x_scales=J),
                                  dict(ws=H), dict(ws=I), dict(h=G), dict(out=D), dict(x_codes=B)]),
    (bwd, abi.CONVIMG_ERR_SHAPE, [dict(M=-1), dict(N=0), dict(K=0), dict(lddy=47), dict(ldx=63), dict(adapters=0),
                                  dict(rank=0)]),
    (bwd, abi.CONVIMG_ERR_DTYPE, [dict(dy_dtype=KEPT), dict(x_dtype=MX), dict(x_dtype=5), dict(a_dtype=KEPT),
                                  dict(dx_dtype=MX)]),
    (bwd, abi.CONVIMG_ERR_RANGE, [dict(rank=4097), dict(N=1 << 25, lddy=1 << 25), dict(M=1, K=1 << 25, ldx=1 << 25),
                                  dict(M=1 << 26)]),
    (bwd, abi.CONVIMG_ERR_NULL, [dict([(n, None)]) for n in ("dy", "x", "wt_codes", "wt_scales", "down", "up", "scale", "ids",
                                                             "h", "dx", "ddown", "dup", "ws")]
     + [dict(x_dtype=KEPT, x_scales=None)]),
    (bwd, abi.CONVIMG_ERR_ALIGN, [dict(wt_codes=C + 8), dict(wt_scales=D + 2), dict(ws=M + 8),
                                  dict(x_dtype=KEPT, x=B + 8, x_scales=N), dict(x_dtype=KEPT, x_scales=N + 2)]),
    (bwd, abi.CONVIMG_ERR_WORKSPACE, [dict(ws_bytes=256)]),
    (bwd, abi.CONVIMG_ERR_ALIAS, [dict(dx=A), dict(dx=B), dict(ddown=E), dict(dup=F), dict(dup=K + 4), dict(ws=J), dict(ws=I),
                                  dict(ddown=H), dict(dup=G), dict(x_dtype=KEPT, x_scales=J + 4)]),
]


@pytest.mark.parametrize("fn,status,calls", CASES, ids=lambda v: getattr(v, "__name__", None) or "")
def test_refusals(fn, status, calls):
    for kw in calls:
        assert fn(**kw) == status, "%s(%s)" % (fn.__name__, kw)


def test_sizes():
    assert abi.mxint8_bytes(5, 33) == (0, 5 * 64, 5 * 4)
    assert abi.mxint8_bytes(0, 1) == (0, 0, 0)
    assert abi.mxint8_bytes(7, 129) == (0, 7 * 160, 7 * 8)
    assert abi.mxint8_bytes(1 << 20, 1 << 12) == (0, 1 << 32, 1 << 27)      # past 2 GiB
    assert abi.mxint8_bytes(3, 0)[0] == abi.CONVIMG_ERR_SHAPE
    assert abi.mxint8_bytes(1 << 31, 1)[0] == abi.CONVIMG_ERR_RANGE
    assert abi.mxfp4_linear_adapters_workspace(8, 48, 64, 0, 4, BF16)[0] == abi.CONVIMG_ERR_SHAPE
    assert abi.mxfp4_linear_adapters_workspace(8, 48, 64, 3, 4, MX)[0] == abi.CONVIMG_ERR_DTYPE
    assert abi.mxfp4_linear_adapters_bwd_workspace(8, 48, 64, 3, 0)[0] == abi.CONVIMG_ERR_SHAPE
    assert abi.mxfp4_linear_adapters_bwd_workspace(8, (1 << 25) - 1, 64, 3, 64)[0] == 0
    # 2^18 tiles of columns by 64 chunks of ranks: the gradients' launch would hold 2^32 threads
    assert abi.mxfp4_linear_adapters_bwd_workspace(8, (1 << 25) - 1, 64, 3, 4096)[0] == abi.CONVIMG_ERR_RANGE
    for m in (1, 8, 100, 5000):      # at least the packed rows and h
        rc, n = abi.mxfp4_linear_adapters_workspace(m, 48, 64, 3, 4, FP16)
        assert rc == 0 and n >= m * 16
        rc, n = abi.mxfp4_linear_adapters_bwd_workspace(m, 48, 64, 3, 4)
        assert rc == 0 and n >= m * (24 + 16)


def test_empty_batches_need_no_data():
    assert quant(rows=0, x=None) == 0
    assert deq(rows=0, out=None) == 0
    assert ln(rows=0, x=None, y=None, codes=None, scales=None, rstd=None) == 0
    assert fwd(M=0, x=None, out=None, ids=None) == 0


def test_wrappers_refuse_host_tensors():
    x = torch.zeros(4, 64)
    q = cim.Mxint8Tensor(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 4, dtype=torch.uint8), 4, 64)
    w = cim.Mxfp4Tensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8), 4, 64)
    ad = cim.Adapters(torch.zeros(2, 3, 64), torch.zeros(2, 3, 4), torch.ones(2))
    ids = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: cim.mxint8_quantize_nhwc(x), lambda: cim.mxint8_dequantize_nhwc(q, torch.float32),
                 lambda: cim.layer_norm_mxint8_nhwc(x), lambda: cim.layer_norm_bwd_mxint8_nhwc(x, q, None, x[:, 0]),
                 lambda: cim.mxfp4_linear_bwd_nhwc(x, q, x), lambda: cim.mxfp4_linear_adapters_nhwc(x, w, None, ad, ids),
                 lambda: cim.mxfp4_linear_adapters_bwd_nhwc(x, x, w, ad, ids, x)):
        with pytest.raises(ValueError):
            call()


class Wide(Machine):
    """test_row_wrappers_host's machine with the entry points of this file."""

    def __init__(self, monkeypatch):
        super().__init__(monkeypatch)
        for n in ("quantize8", "dequantize8", "layer_norm_kept", "layer_norm_kept_bwd", "adapters", "adapters_bwd"):
            monkeypatch.setattr(R._fast, n, lambda *a: None, raising=False)
        for n in ("mxint8_quantize", "mxint8_dequantize", "layer_norm_fwd_mxint8", "layer_norm_bwd_mxint8",
                  "mxfp4_linear_bwd_mxint8", "mxfp4_linear_adapters_fwd", "mxfp4_linear_adapters_bwd"):
            monkeypatch.setattr(R._lib, n, self.entry(n), raising=False)
        assert isinstance(R._lib, types.SimpleNamespace)


@pytest.fixture
def machine(monkeypatch):
    return Wide(monkeypatch)


def operands():
    x, w, dy = dev(torch.ones(300, 256)), dev(torch.ones(128, 256)), dev(torch.ones(300, 128))
    q4 = R.Mxfp4Tensor(dev(torch.zeros(128, 128, dtype=torch.uint8)), dev(torch.zeros(2, 128, 4, dtype=torch.uint8)), 128, 256)
    t4 = R.Mxfp4Tensor(dev(torch.zeros(256, 64, dtype=torch.uint8)), dev(torch.zeros(1, 256, 4, dtype=torch.uint8)), 256, 128)
    q8 = R.Mxint8Tensor(dev(torch.zeros(300, 256, dtype=torch.int8)), dev(torch.zeros(300, 8, dtype=torch.uint8)), 300, 256)
    ad = R.Adapters(dev(torch.ones(2, 5, 256)), dev(torch.ones(2, 5, 128)), dev(torch.ones(2)))
    return x, w, dy, q4, t4, q8, ad, dev(torch.zeros(300, dtype=torch.int32)), dev(torch.ones(300, 5)), dev(torch.ones(300))


def calls():
    x, w, dy, q4, t4, q8, ad, ids, h, rstd = operands()
    return [lambda **s: R.mxint8_quantize_nhwc(x, **s), lambda **s: R.mxint8_dequantize_nhwc(q8, torch.float32, **s),
            lambda **s: R.layer_norm_mxint8_nhwc(x, **s), lambda **s: R.layer_norm_bwd_mxint8_nhwc(x, q8, None, rstd, **s),
            lambda **s: R.mxfp4_linear_bwd_nhwc(dy, q8, w, **s),
            lambda **s: R.mxfp4_linear_adapters_nhwc(x, q4, None, ad, ids, save=True, **s),
            lambda **s: R.mxfp4_linear_adapters_nhwc(x, q4, None, ad, ids, **s),
            lambda **s: R.mxfp4_linear_adapters_bwd_nhwc(dy, q8, t4, ad, ids, h, **s),
            lambda **s: R.mxfp4_linear_adapters_bwd_nhwc(dy, x, t4, ad, ids, h, **s)]


@pytest.mark.parametrize("k", range(9))
def test_buffers_of_another_stream_are_its_own(machine, k):
    call = calls()[k]
    out = tensors(call(stream=SIDE))
    assert machine.calls[-1][1][-1] == SIDE
    assert machine.made and set(machine.made.values()) == {SIDE}
    assert {(t.data_ptr(), HOME) for t in out} <= set(Dev.recorded)
    assert machine.current == HOME
    machine.made.clear()
    Dev.recorded.clear()
    for s in (None, HOME):
        call(stream=s)
        assert machine.calls[-1][1][-1] == HOME and set(machine.made.values()) == {HOME} and not Dev.recorded


def test_results_have_their_types(machine):
    q = calls()[0]()
    assert isinstance(q, R.Mxint8Tensor) and q.codes.dtype == torch.int8 and q.codes.shape == (300, 256)
    y, kept, rstd = calls()[2]()
    assert isinstance(kept, R.Mxint8Tensor) and rstd.shape == (300,)
    out, kept, h = calls()[5]()
    assert isinstance(kept, R.Mxint8Tensor) and h.shape == (300, 5) and out.shape == (300, 128)
    x, _, dy, _, _, q8, ad, ids, h, _ = operands()
    dx, ddown, dup = R.mxfp4_linear_adapters_bwd_nhwc(dy, q8, None, ad, ids, h)
    args = machine.calls[-1][1]
    assert dx is None and args[7:9] == (None, None) and args[21] is None and ddown.shape == (2, 5, 256) and dup.shape == (2, 5, 128)


def test_wrappers_refuse(machine):
    x, w, dy, q4, t4, q8, ad, ids, h, rstd = operands()
    fwd = lambda x=x, w=q4, b=None, a=ad, i=ids, **k: R.mxfp4_linear_adapters_nhwc(x, w, b, a, i, **k)      # noqa: E731
    back = lambda dy=dy, x=q8, w=t4, a=ad, i=ids, h=h, **k: R.mxfp4_linear_adapters_bwd_nhwc(dy, x, w, a, i, h, **k)      # noqa: E731
    wrong = [lambda: fwd(x=dev(torch.ones(300, 255))), lambda: fwd(b=dev(torch.ones(127))), lambda: fwd(i=dev(torch.zeros(300))),
             lambda: fwd(i=dev(torch.zeros(299, dtype=torch.int32))), lambda: fwd(i=dev(torch.zeros(300, 2, dtype=torch.int32))[:, 0]),
             lambda: fwd(a=ad._replace(down=dev(torch.ones(2, 5, 255)))), lambda: fwd(a=ad._replace(up=dev(torch.ones(2, 4, 128)))),
             lambda: fwd(a=ad._replace(up=dev(torch.ones(3, 5, 128)))), lambda: fwd(a=ad._replace(scale=dev(torch.ones(3)))),
             lambda: fwd(a=ad._replace(scale=None)), lambda: fwd(a=ad._replace(down=dev(torch.ones(2, 256, 5)).transpose(1, 2))),
             lambda: fwd(a=R.Adapters(dev(torch.ones(0, 5, 256)), dev(torch.ones(0, 5, 128)), dev(torch.ones(0)))),
             lambda: back(dy=dev(torch.ones(299, 128))), lambda: back(x=q8._replace(rows=299)), lambda: back(w=q4),
             lambda: back(x=q8._replace(codes=q8.codes.to(torch.uint8))), lambda: back(h=dev(torch.ones(300, 4))),
             lambda: back(h=dev(torch.ones(300, 5).double())), lambda: back(i=dev(torch.zeros(300, dtype=torch.int64))),
             lambda: R.mxint8_dequantize_nhwc(q8._replace(cols=300), torch.float32),
             lambda: R.layer_norm_bwd_mxint8_nhwc(dy, q8, None, rstd), lambda: R.layer_norm_bwd_mxint8_nhwc(x, q8, None, rstd[:9]),
             lambda: R.mxfp4_linear_bwd_nhwc(dy, q8, dev(torch.ones(128, 255))),
             lambda: R.mxfp4_linear_bwd_nhwc(dev(torch.ones(299, 128)), q8, w)]
    for k, call in enumerate(wrong):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d" % k)
    for call in (lambda: fwd(a=ad._replace(up=ad.up.to(torch.bfloat16))), lambda: fwd(out_dtype=torch.int32),
                 lambda: fwd(x=dev(torch.ones(300, 256).double())), lambda: back(dx_dtype=torch.float64),
                 lambda: R.mxint8_quantize_nhwc(dev(torch.ones(3, 4, dtype=torch.int32))),
                 lambda: R.mxint8_dequantize_nhwc(q8, torch.int8)):
        with pytest.raises(TypeError):
            call()
    assert not machine.calls


MANY = (1 << 32) + 5      # 5 in 32 bits


def many8(rows, cols):
    return R.Mxint8Tensor(far(rows, -(-cols // 32) * 32, dtype=torch.int8), far(rows, -(-cols // 128) * 4, dtype=torch.uint8), rows, cols)


@pytest.mark.parametrize("call", [
    lambda: R.mxint8_quantize_nhwc(far(MANY, 32)), lambda: R.mxint8_quantize_nhwc(far(1, MANY)),
    lambda: R.mxint8_dequantize_nhwc(many8(MANY, 32), torch.bfloat16), lambda: R.mxint8_dequantize_nhwc(many8(2, MANY), torch.bfloat16),
    lambda: R.layer_norm_mxint8_nhwc(far(MANY, 4)),
    lambda: R.layer_norm_bwd_mxint8_nhwc(far(MANY, 32), many8(MANY, 32), None, far(MANY, dtype=torch.float32)),
    lambda: R.mxfp4_linear_adapters_nhwc(far(MANY, 32), None, None, None, None),
    lambda: R.mxfp4_linear_adapters_bwd_nhwc(far(MANY, 32), None, None, None, None, None)], ids=range(8))
def test_sizes_past_the_library_s_32_bits_are_refused(machine, call):
    with pytest.raises(RuntimeError, match="status %d" % abi.CONVIMG_ERR_RANGE):
        call()
    assert not machine.calls


def test_uncommon_calls_are_left_to_python():
    R._torch or R._setup()
    f = R._fast
    x, w, dy, q4, t4, q8, ad, ids, h, rstd = operands()      # host memory
    plain = lambda q: tuple(torch.Tensor(t) if isinstance(t, Dev) else t for t in q)      # noqa: E731
    for call in (lambda: f.quantize8(x), lambda: f.dequantize8(plain(q8), torch.float32), lambda: f.dequantize8(7, torch.float32),
                 lambda: f.dequantize8((1, 2, "a", None), torch.float32), lambda: f.layer_norm_kept(x, None, None, 1e-5, None),
                 lambda: f.layer_norm_kept_bwd(x, q8, None, rstd, None), lambda: f.linear_bwd(dy, q8, w, None),
                 lambda: f.adapters(x, q4, None, ad, ids, None, False), lambda: f.adapters(None, None, None, None, None, None, True),
                 lambda: f.adapters_bwd(dy, q8, t4, ad, ids, h, None), lambda: f.adapters_bwd(dy, x, None, (1, 2), ids, h, None)):
        assert call() is None
    for call in (lambda: f.quantize8(), lambda: f.adapters(x), lambda: f.adapters_bwd(x, x)):
        with pytest.raises(TypeError):
            call()
