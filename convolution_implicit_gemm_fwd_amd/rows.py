"""Torch wrappers of the row operators: layer norm, MXFP4 and the quantised
linear layer, on channels-last tensors [..., C].

Every dimension before the last is a row index; the last dimension must be
contiguous and the rows evenly spaced (any NHWC tensor, or a column slice of
a matrix).  Calls run on ``stream`` (default: torch's current stream of the
first tensor's device) without waiting; torch supplies device memory and the
stream only.
"""
from __future__ import annotations

from typing import NamedTuple

from . import abi
from .abi import CONVIMG_BF16, CONVIMG_FP16, CONVIMG_FP32, CONVIMG_MXFP4


class Mxfp4Tensor(NamedTuple):
    """Packed rows: uint8 codes [rows, ceil(cols/32)*16] and uint8 scales
    [ceil(cols/128), rows, 4] (include/convimg.h, mxfp4_quantize)."""
    codes: object
    scales: object
    rows: int
    cols: int


_codes = {}


def _dtype(t, what):
    if not _codes:
        import torch
        _codes.update({torch.bfloat16: CONVIMG_BF16, torch.float32: CONVIMG_FP32, torch.float16: CONVIMG_FP16})
    c = _codes.get(t)
    if c is None:
        raise TypeError("%s must be bfloat16, float16 or float32" % what)
    return c


def _rows_of(t, what):
    """(rows, columns, elements from row to row) of a tensor [..., C]."""
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % what)
    shape, strides = t.shape, t.stride()
    d = len(shape)
    if d == 0 or shape[-1] == 0:
        raise ValueError("%s must be [..., C] with C > 0" % what)
    cols = shape[-1]
    if strides[-1] != 1 and cols != 1:
        raise ValueError("the last dimension of %s must be contiguous" % what)
    if d == 2:
        rows, ld = shape[0], strides[0]
    else:
        rows, ld = 1, 0
        for k in range(d - 2, -1, -1):
            if shape[k] == 1:
                continue
            if rows == 1:
                ld = strides[k]
            elif rows and shape[k] and strides[k] != ld * rows:
                raise ValueError("the rows of %s must be evenly spaced" % what)
            rows *= shape[k]
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError("the rows of %s must not overlap" % what)
    return rows, cols, ld


def _param(t, cols, like, what):
    import torch

    if t is None:
        return None
    if t.dtype != torch.float32 or t.device != like.device or t.dim() != 1 or t.shape[0] != cols \
            or not t.is_contiguous():
        raise ValueError("%s must be a contiguous float32 tensor of %d values on the input's device" % (what, cols))
    return t.data_ptr()


class _Call:
    """The device and stream of one call, and the buffers it allocates."""

    def __init__(self, t, stream):
        import torch

        self.torch, self.device = torch, t.device
        self.current = torch.cuda.current_stream(t.device).cuda_stream
        self.stream = self.current if stream is None else stream
        self.fresh = []

    def empty(self, shape, dtype):
        t = self.torch.empty(shape, dtype=dtype, device=self.device)
        if self.stream != self.current:
            self.fresh.append(t)
        return t

    def run(self, fn, *args):
        torch = self.torch
        if torch.cuda.current_device() == self.device.index:
            rc = fn(*args, self.stream)
        else:
            with torch.cuda.device(self.device):
                rc = fn(*args, self.stream)
        if rc != 0:
            raise RuntimeError("%s failed: %s (status %d)" % (fn.__name__, abi.conv2d_strerror(rc), rc))
        if self.fresh:
            # allocated on torch's current stream, used on another: the
            # allocator must not hand the memory out before that stream is done
            ext = torch.cuda.ExternalStream(self.stream, device=self.device)
            for t in self.fresh:
                t.record_stream(ext)


def _check(rc, what):
    if rc != 0:
        raise RuntimeError("%s failed: %s (status %d)" % (what, abi.conv2d_strerror(rc), rc))


def _same_device(like, **tensors):
    for name, t in tensors.items():
        if t.device != like.device:
            raise ValueError("%s must be on the device of the other tensors" % name)


def layer_norm_nhwc(x, gamma=None, beta=None, eps=1e-5, out_dtype=None, stats=False, stream=None):
    """y = (x - mean) / sqrt(var + eps) * gamma + beta over the last dimension.

    x: [..., C] bfloat16, float16 or float32; gamma, beta: float32 [C] or
    None.  Returns y, contiguous, of x's shape in ``out_dtype`` (default: x's);
    with ``stats`` (y, mean, rstd), the float32 row statistics that
    ``layer_norm_bwd_nhwc`` takes, of x's shape without the last dimension.
    """
    rows, cols, ld = _rows_of(x, "x")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    xd, yd = _dtype(x.dtype, "x"), _dtype(out_dtype, "out_dtype")
    g, b = _param(gamma, cols, x, "gamma"), _param(beta, cols, x, "beta")
    c = _Call(x, stream)
    y = c.empty(x.shape, out_dtype)
    mean = rstd = None
    if stats:
        mean, rstd = c.empty(x.shape[:-1], c.torch.float32), c.empty(x.shape[:-1], c.torch.float32)
    c.run(abi.layer_norm_fwd, x.data_ptr(), ld, g, b, rows, cols, eps, xd, yd, y.data_ptr(),
          mean.data_ptr() if stats else None, rstd.data_ptr() if stats else None)
    return (y, mean, rstd) if stats else y


def _packed(c, rows, cols):
    nb = -(-cols // 32)
    return Mxfp4Tensor(c.empty((rows, nb * 16), c.torch.uint8), c.empty((-(-nb // 4), rows, 4), c.torch.uint8),
                       rows, cols)


def layer_norm_mxfp4_nhwc(x, gamma=None, beta=None, eps=1e-5, stream=None):
    """layer_norm_nhwc with its result quantised to MXFP4 rows: an
    ``Mxfp4Tensor``, the input of ``mxfp4_linear_nhwc``."""
    rows, cols, ld = _rows_of(x, "x")
    xd = _dtype(x.dtype, "x")
    g, b = _param(gamma, cols, x, "gamma"), _param(beta, cols, x, "beta")
    c = _Call(x, stream)
    q = _packed(c, rows, cols)
    c.run(abi.layer_norm_fwd_mxfp4, x.data_ptr(), ld, g, b, rows, cols, eps, xd, q.codes.data_ptr(),
          q.scales.data_ptr(), None, None)
    return q


def layer_norm_bwd_nhwc(dy, x, gamma, mean, rstd, dx_dtype=None, stream=None):
    """(dx, dgamma, dbeta): gradients of layer_norm_nhwc.

    dy, x: [..., C] of one shape, each bfloat16, float16 or float32; gamma:
    float32 [C] or None; mean, rstd: the forward's statistics.  dx: contiguous,
    in ``dx_dtype`` (default: x's dtype); dgamma and dbeta: float32 [C].
    """
    rows, cols, ld = _rows_of(x, "x")
    if dy.shape != x.shape:
        raise ValueError("dy must have x's shape")
    _, _, ldy = _rows_of(dy, "dy")
    _same_device(x, dy=dy)
    dx_dtype = x.dtype if dx_dtype is None else dx_dtype
    dd, xd, od = _dtype(dy.dtype, "dy"), _dtype(x.dtype, "x"), _dtype(dx_dtype, "dx_dtype")
    g = _param(gamma, cols, x, "gamma")
    m, r = _param(mean.reshape(-1), rows, x, "mean"), _param(rstd.reshape(-1), rows, x, "rstd")
    c = _Call(x, stream)
    rc, need = abi.layer_norm_bwd_workspace(rows, cols)
    _check(rc, "layer_norm_bwd_workspace")
    f32 = c.torch.float32
    dx, dgamma, dbeta = c.empty(x.shape, dx_dtype), c.empty((cols,), f32), c.empty((cols,), f32)
    ws = c.empty((need,), c.torch.uint8)
    c.run(abi.layer_norm_bwd, dy.data_ptr(), ldy, x.data_ptr(), ld, g, m, r, rows, cols, dd, xd, od, dx.data_ptr(),
          dgamma.data_ptr(), dbeta.data_ptr(), ws.data_ptr(), need)
    return dx, dgamma, dbeta


def mxfp4_quantize_nhwc(x, transpose=False, stream=None):
    """x [..., C] as MXFP4 rows (an ``Mxfp4Tensor``); ``transpose``: the rows of
    its transpose, so that blocks of 32 run down the columns of x."""
    rows, cols, ld = _rows_of(x, "x")
    xd = _dtype(x.dtype, "x")
    c = _Call(x, stream)
    q = _packed(c, cols, rows) if transpose else _packed(c, rows, cols)
    c.run(abi.mxfp4_quantize, x.data_ptr(), ld, rows, cols, xd, 1 if transpose else 0, q.codes.data_ptr(),
          q.scales.data_ptr())
    return q


def _check_packed(q, what):
    import torch

    nb = -(-q.cols // 32)
    for t, shape in ((q.codes, (q.rows, nb * 16)), (q.scales, (-(-nb // 4), q.rows, 4))):
        if t.dtype != torch.uint8 or not t.is_cuda or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError("%s is not a packed operand of %d rows and %d columns" % (what, q.rows, q.cols))


def mxfp4_dequantize_nhwc(q, dtype, stream=None):
    """The values [rows, cols] that packed rows stand for, in ``dtype``."""
    _check_packed(q, "q")
    d = _dtype(dtype, "dtype")
    c = _Call(q.codes, stream)
    out = c.empty((q.rows, q.cols), dtype)
    c.run(abi.mxfp4_dequantize, q.codes.data_ptr(), q.scales.data_ptr(), q.rows, q.cols, d, out.data_ptr())
    return out


def mxfp4_linear_nhwc(x, w, bias=None, out_dtype=None, stream=None):
    """out[..., n] = sum_k Q(x)[..., k] * w[n, k] + bias[n], a 1x1 convolution on
    4-bit operands.

    x: [..., K] dense (quantised by the call) or an ``Mxfp4Tensor`` of K
    columns; w: an ``Mxfp4Tensor`` of N rows and K columns; bias: float32 [N] or
    None.  out: contiguous, in ``out_dtype`` (default: x's dtype, bfloat16 for packed x).
    """
    _check_packed(w, "w")
    like = w.codes
    c = _Call(like, stream)
    torch = c.torch
    if isinstance(x, Mxfp4Tensor):
        _check_packed(x, "x")
        M, K, ld, xd, shape = x.rows, x.cols, x.cols, CONVIMG_MXFP4, (x.rows,)
        xp, sp = x.codes.data_ptr(), x.scales.data_ptr()
        _same_device(like, x=x.codes)
        out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    else:
        M, K, ld = _rows_of(x, "x")
        xd, shape, xp, sp = _dtype(x.dtype, "x"), x.shape[:-1], x.data_ptr(), None
        _same_device(like, x=x)
        out_dtype = x.dtype if out_dtype is None else out_dtype
    if K != w.cols:
        raise ValueError("x has %d columns, w %d" % (K, w.cols))
    N = w.rows
    od = _dtype(out_dtype, "out_dtype")
    b = _param(bias, N, like, "bias")
    rc, need = abi.mxfp4_linear_workspace(M, N, K, xd)
    _check(rc, "mxfp4_linear_workspace")
    out = c.empty((*shape, N), out_dtype)
    ws = c.empty((need,), torch.uint8) if need else None
    c.run(abi.mxfp4_linear_fwd, xp, ld, sp, xd, like.data_ptr(), w.scales.data_ptr(), b, M, N, K, od, out.data_ptr(),
          ws.data_ptr() if need else None, need)
    return out


def mxfp4_linear_bwd_nhwc(dy, x, w, dx_dtype=None, stream=None):
    """(dx, dw, db): gradients of the linear layer on 4-bit operands.

    dy: [..., N]; x: [..., K] and w: [N, K], the forward input and weights
    before quantisation, of one dtype.  dx: x's shape in ``dx_dtype`` (default:
    x's dtype); dw: float32 [N, K]; db: float32 [N].
    """
    M, N, ldy = _rows_of(dy, "dy")
    mx, K, ldx = _rows_of(x, "x")
    if w.dim() != 2 or mx != M or dy.shape[:-1] != x.shape[:-1] or tuple(w.shape) != (N, K):
        raise ValueError("dy must be [..., N], x [..., K] and w [N, K]")
    if x.dtype != w.dtype:
        raise TypeError("x and w must have one dtype")
    _, _, ldw = _rows_of(w, "w")
    _same_device(dy, x=x, w=w)
    dx_dtype = x.dtype if dx_dtype is None else dx_dtype
    dd, xd, od = _dtype(dy.dtype, "dy"), _dtype(x.dtype, "x"), _dtype(dx_dtype, "dx_dtype")
    rc, need = abi.mxfp4_linear_bwd_workspace(M, N, K)
    _check(rc, "mxfp4_linear_bwd_workspace")
    c = _Call(dy, stream)
    f32 = c.torch.float32
    dx, dw, db = c.empty(x.shape, dx_dtype), c.empty((N, K), f32), c.empty((N,), f32)
    ws = c.empty((need,), c.torch.uint8)
    c.run(abi.mxfp4_linear_bwd, dy.data_ptr(), ldy, dd, x.data_ptr(), ldx, w.data_ptr(), ldw, xd, M, N, K, od,
          dx.data_ptr(), dw.data_ptr(), db.data_ptr(), ws.data_ptr(), need)
    return dx, dw, db
