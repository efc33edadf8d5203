"""Torch wrappers of the row operators: layer norm, MXFP4 and the quantised
linear layer, low-rank adapters beside it and activations kept in 8 bits, on
channels-last tensors [..., C].

Every dimension before the last is a row index; the last dimension must be
contiguous and the rows evenly spaced (any NHWC tensor, or a column slice of
a matrix).  Calls run on ``stream`` (a stream's handle; default: torch's current
stream of the first tensor's device) without waiting; torch supplies device
memory and the stream only.  A call on another stream than the current one is
made as under ``torch.cuda.stream``: its outputs and workspace come from that
stream's memory, and the caller orders that stream behind whatever made the
inputs, keeps the inputs until it has run the call, and orders what reads the
outputs behind it.

A small call costs the host more than the GPU (a launch is about 3 us, the
kernel of one 4096-wide token 2 us), so the common case (tensors as they
should be, on the current device and stream) takes its whole way in compiled
code (csrc/rows_ext.cpp); everything else, errors included, is handled here.
"""
from __future__ import annotations

from functools import lru_cache
from typing import NamedTuple

from . import abi
from .abi import CONVIMG_BF16, CONVIMG_FP16, CONVIMG_FP32, CONVIMG_MXFP4, CONVIMG_MXINT8


class Mxfp4Tensor(NamedTuple):
    """Packed rows: uint8 codes [rows, ceil(cols/32)*16] and uint8 scales
    [ceil(cols/128), rows, 4] (include/convimg.h, mxfp4_quantize)."""
    codes: object
    scales: object
    rows: int
    cols: int


class Mxint8Tensor(NamedTuple):
    """Activations kept in 8 bits: int8 codes [rows, cols rounded up to 32] and
    uint8 scales [rows, 4 * ceil(cols/128)] (include/convimg.h, mxint8_quantize)."""
    codes: object
    scales: object
    rows: int
    cols: int


class Adapters(NamedTuple):
    """Low-rank adapters of one rank r: down [G, r, K] and up [G, r, N],
    contiguous, of one dtype (bfloat16, float16 or float32), scale float32 [G].
    Adapter g adds scale[g] * up[g]^T (down[g] x) to a layer's output."""
    down: object
    up: object
    scale: object


_torch = None
_new = tuple.__new__


def _setup():
    """torch, the loaded library and what every call takes from them."""
    global _torch, _fast, _lib, _codes, _f32, _u8, _i8, _i32, _device, _stream, _empty
    import ctypes

    import torch

    _lib = abi.load()
    try:
        from . import _rows as _fast
    except ImportError as e:
        raise abi.LibraryMissing(
            "_rows.so, the row operators' torch module, is not built or does not load (%s); build it with "
            "`python -m convolution_implicit_gemm_fwd_amd.build`" % e) from e
    for name in ("layer_norm_fwd", "layer_norm_fwd_mxfp4", "layer_norm_bwd", "layer_norm_bwd_workspace",
                 "mxfp4_quantize", "mxfp4_dequantize", "mxfp4_linear_fwd", "mxfp4_linear_workspace",
                 "mxfp4_linear_bwd", "mxfp4_linear_bwd_workspace", "mxint8_quantize", "mxint8_dequantize",
                 "layer_norm_fwd_mxint8", "layer_norm_bwd_mxint8", "mxfp4_linear_bwd_mxint8",
                 "mxfp4_linear_adapters_fwd", "mxfp4_linear_adapters_workspace", "mxfp4_linear_adapters_bwd",
                 "mxfp4_linear_adapters_bwd_workspace"):
        _fast.bind(name, ctypes.cast(getattr(_lib, name), ctypes.c_void_p).value)
    _codes = {torch.bfloat16: CONVIMG_BF16, torch.float32: CONVIMG_FP32, torch.float16: CONVIMG_FP16}
    _f32, _u8, _i8, _i32 = torch.float32, torch.uint8, torch.int8, torch.int32
    _device = torch.cuda.current_device
    _empty = torch.empty       # (sizes as separate numbers: 0.3 us less than as a tuple)
    # the current stream's handle: the raw getter, where torch has it, makes no Stream object (0.1 us, not 1.9)
    _stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) \
        or (lambda index: torch.cuda.current_stream(index).cuda_stream)
    _torch = torch


def _query(fn):
    """A workspace's bytes by sizes and types."""
    @lru_cache(maxsize=1024)
    def bytes_of(*args):
        rc, n = fn(*args)
        if rc:
            _fail(fn.__name__, rc)
        return n
    return bytes_of


_norm_bwd_bytes = _query(abi.layer_norm_bwd_workspace)
_linear_bytes = _query(abi.mxfp4_linear_workspace)
_linear_bwd_bytes = _query(abi.mxfp4_linear_bwd_workspace)
_adapters_bytes = _query(abi.mxfp4_linear_adapters_workspace)
_adapters_bwd_bytes = _query(abi.mxfp4_linear_adapters_bwd_workspace)


def _dtype(t, what):
    c = _codes.get(t)
    if c is None:
        raise TypeError("%s must be bfloat16, float16 or float32" % what)
    return c


def _fits(rows, cols, what):
    """Counts as the library's ints: ctypes would pass their lower 32 bits."""
    if rows > 0x7fffffff or cols > 0x7fffffff:
        rc = abi.CONVIMG_ERR_RANGE
        raise RuntimeError("%s has %d rows of %d columns: %s (status %d)" % (what, rows, cols, abi.conv2d_strerror(rc), rc))


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
    _fits(rows, cols, what)
    return rows, cols, ld


def _param(t, n, device, what):
    """The address of a float32 vector of n values, None for None."""
    if t is None:
        return None
    if t.dtype is not _f32 or t.device != device or t.shape != (n,) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous float32 tensor of %d values on the input's device" % (what, n))
    return t.data_ptr()


def _like(t, dtype):
    """An uninitialised contiguous tensor of t's shape."""
    if t.is_contiguous():
        return _torch.empty_like(t, dtype=dtype)
    return _empty(*t.shape, dtype=dtype, device=t.device)


def _elsewhere(device, f, *args):
    """The call with the tensors' device made the current one."""
    with _torch.cuda.device(device):
        return f(*args)


def _fail(name, rc):
    raise RuntimeError("%s failed: %s (status %d)" % (name, abi.conv2d_strerror(rc), rc))


def _on(stream, t, f, *args):
    """The call on the stream of this handle, where that is not the current one
    of t's device with the stream made the current one: a block of the present
    current stream's memory may be in use by work that is still queued there.
    The results go back to that stream, so their memory is not used again
    before it is past them."""
    if not t.is_cuda:
        return f(*args)        # (refused there)
    device = t.device
    if _device() != device.index:
        return _elsewhere(device, _on, stream, t, f, *args)
    if stream == _stream(device.index):
        return f(*args)
    # (set and set back: 4 us less than torch.cuda.stream, which looks up the device and the stream twice)
    home = _torch.cuda.current_stream(device.index)
    _torch.cuda.set_stream(_torch.cuda.ExternalStream(stream, device=device))
    try:
        r = f(*args)
    finally:
        _torch.cuda.set_stream(home)
    _record(r, home)
    return r


def _record(r, stream):
    if isinstance(r, _torch.Tensor):
        r.record_stream(stream)
    elif isinstance(r, tuple):
        for o in r:
            _record(o, stream)


def _same_device(device, t, what):
    if t.device != device:
        raise ValueError("%s must be on the device of the other tensors" % what)


def _stats(x):
    """(mean, rstd) for the rows of x to write, and their addresses."""
    mean = _empty(*x.shape[:-1], dtype=_f32, device=x.device) if x.dim() > 1 else _empty((), dtype=_f32, device=x.device)
    rstd = _torch.empty_like(mean)
    return mean, rstd, mean.data_ptr(), rstd.data_ptr()


def layer_norm_nhwc(x, gamma=None, beta=None, eps=1e-5, out_dtype=None, stats=False, stream=None):
    """y = (x - mean) / sqrt(var + eps) * gamma + beta over the last dimension.

    x: [..., C] bfloat16, float16 or float32; gamma, beta: float32 [C] or
    None.  Returns y, contiguous, of x's shape in ``out_dtype`` (default: x's);
    with ``stats`` (y, mean, rstd), the float32 row statistics that
    ``layer_norm_bwd_nhwc`` takes, of x's shape without the last dimension.
    """
    if _torch is None:
        _setup()
    if stream is not None:
        return _on(stream, x, layer_norm_nhwc, x, gamma, beta, eps, out_dtype, stats)
    r = _fast.layer_norm(x, gamma, beta, eps, out_dtype, stats)
    if r is not None:
        return r
    rows, cols, ld = _rows_of(x, "x")
    dev = x.device
    if _device() != dev.index:
        return _elsewhere(dev, layer_norm_nhwc, x, gamma, beta, eps, out_dtype, stats)
    if out_dtype is None:
        out_dtype = x.dtype
    xd, yd = _dtype(x.dtype, "x"), _dtype(out_dtype, "out_dtype")
    g, b = _param(gamma, cols, dev, "gamma"), _param(beta, cols, dev, "beta")
    y = _like(x, out_dtype)
    mean, rstd, mp, rp = _stats(x) if stats else (None,) * 4
    rc = _lib.layer_norm_fwd(x.data_ptr(), ld, g, b, rows, cols, eps, xd, yd, y.data_ptr(), mp, rp,
                             _stream(dev.index))
    if rc:
        _fail("layer_norm_fwd", rc)
    return (y, mean, rstd) if stats else y


def _packed(device, rows, cols):
    nb = -(-cols // 32)
    return Mxfp4Tensor(_empty(rows, nb * 16, dtype=_u8, device=device),
                       _empty(-(-nb // 4), rows, 4, dtype=_u8, device=device), rows, cols)


def layer_norm_mxfp4_nhwc(x, gamma=None, beta=None, eps=1e-5, stream=None, stats=False):
    """layer_norm_nhwc with its result quantised to MXFP4 rows: an
    ``Mxfp4Tensor``, the input of ``mxfp4_linear_nhwc``; with ``stats``
    (that, mean, rstd), the statistics as ``layer_norm_nhwc`` gives them."""
    if _torch is None:
        _setup()
    if stream is not None:
        return _on(stream, x, layer_norm_mxfp4_nhwc, x, gamma, beta, eps, None, stats)
    if not stats:
        r = _fast.layer_norm_mxfp4(x, gamma, beta, eps)
        if r is not None:
            return _new(Mxfp4Tensor, r)
    rows, cols, ld = _rows_of(x, "x")
    dev = x.device
    if _device() != dev.index:
        return _elsewhere(dev, layer_norm_mxfp4_nhwc, x, gamma, beta, eps, None, stats)
    xd = _dtype(x.dtype, "x")
    g, b = _param(gamma, cols, dev, "gamma"), _param(beta, cols, dev, "beta")
    q = _packed(dev, rows, cols)
    mean, rstd, mp, rp = _stats(x) if stats else (None,) * 4
    rc = _lib.layer_norm_fwd_mxfp4(x.data_ptr(), ld, g, b, rows, cols, eps, xd, q.codes.data_ptr(),
                                   q.scales.data_ptr(), mp, rp, _stream(dev.index))
    if rc:
        _fail("layer_norm_fwd_mxfp4", rc)
    return (q, mean, rstd) if stats else q


def layer_norm_bwd_nhwc(dy, x, gamma, mean, rstd, dx_dtype=None, stream=None):
    """(dx, dgamma, dbeta): gradients of layer_norm_nhwc.

    dy, x: [..., C] of one shape, each bfloat16, float16 or float32; gamma:
    float32 [C] or None; mean, rstd: the forward's statistics, float32 in any
    layout (copied if they are not contiguous).  dx: contiguous, in
    ``dx_dtype`` (default: x's dtype); dgamma and dbeta: float32 [C].
    """
    if _torch is None:
        _setup()
    if stream is not None:
        return _on(stream, x, layer_norm_bwd_nhwc, dy, x, gamma, mean, rstd, dx_dtype)
    r = _fast.layer_norm_bwd(dy, x, gamma, mean, rstd, dx_dtype)
    if r is not None:
        return r
    rows, cols, ld = _rows_of(x, "x")
    dev = x.device
    if dy.shape != x.shape:
        raise ValueError("dy must have x's shape")
    ldy = _rows_of(dy, "dy")[2]
    _same_device(dev, dy, "dy")
    if _device() != dev.index:
        return _elsewhere(dev, layer_norm_bwd_nhwc, dy, x, gamma, mean, rstd, dx_dtype)
    if dx_dtype is None:
        dx_dtype = x.dtype
    dd, xd, od = _dtype(dy.dtype, "dy"), _dtype(x.dtype, "x"), _dtype(dx_dtype, "dx_dtype")
    g = _param(gamma, cols, dev, "gamma")
    # (held until the call is made: each may be a copy)
    mean, rstd = mean.reshape(-1).contiguous(), rstd.reshape(-1).contiguous()
    m, r = _param(mean, rows, dev, "mean"), _param(rstd, rows, dev, "rstd")
    need = _norm_bwd_bytes(rows, cols)
    dx = _like(x, dx_dtype)
    dgamma, dbeta = _empty(cols, dtype=_f32, device=dev), _empty(cols, dtype=_f32, device=dev)
    ws = _empty(need, dtype=_u8, device=dev)
    rc = _lib.layer_norm_bwd(dy.data_ptr(), ldy, x.data_ptr(), ld, g, m, r, rows, cols, dd, xd, od, dx.data_ptr(),
                             dgamma.data_ptr(), dbeta.data_ptr(), ws.data_ptr(), need,
                             _stream(dev.index))
    if rc:
        _fail("layer_norm_bwd", rc)
    return dx, dgamma, dbeta


def mxfp4_quantize_nhwc(x, transpose=False, stream=None):
    """x [..., C] as MXFP4 rows (an ``Mxfp4Tensor``); ``transpose``: the rows of
    its transpose, so that blocks of 32 run down the columns of x."""
    if _torch is None:
        _setup()
    if stream is not None:
        return _on(stream, x, mxfp4_quantize_nhwc, x, transpose)
    r = _fast.quantize(x, transpose)
    if r is not None:
        return _new(Mxfp4Tensor, r)
    rows, cols, ld = _rows_of(x, "x")
    dev = x.device
    if _device() != dev.index:
        return _elsewhere(dev, mxfp4_quantize_nhwc, x, transpose)
    xd = _dtype(x.dtype, "x")
    q = _packed(dev, cols, rows) if transpose else _packed(dev, rows, cols)
    rc = _lib.mxfp4_quantize(x.data_ptr(), ld, rows, cols, xd, 1 if transpose else 0, q.codes.data_ptr(),
                             q.scales.data_ptr(), _stream(dev.index))
    if rc:
        _fail("mxfp4_quantize", rc)
    return q


def _check_packed(q, what):
    codes, scales, rows, cols = q
    nb = -(-cols // 32)
    if codes.dtype is not _u8 or scales.dtype is not _u8 or not codes.is_cuda or codes.device != scales.device \
            or codes.shape != (rows, nb * 16) or scales.shape != (-(-nb // 4), rows, 4) \
            or not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError("%s is not a packed operand of %d rows and %d columns" % (what, rows, cols))
    _fits(rows, cols, what)


def mxfp4_dequantize_nhwc(q, dtype, stream=None):
    """The values [rows, cols] that packed rows stand for, in ``dtype``."""
    if _torch is None:
        _setup()
    if stream is not None:
        return _on(stream, q[0], mxfp4_dequantize_nhwc, q, dtype)
    r = _fast.dequantize(q, dtype)
    if r is not None:
        return r
    _check_packed(q, "q")
    d = _dtype(dtype, "dtype")
    codes, scales, rows, cols = q
    dev = codes.device
    if _device() != dev.index:
        return _elsewhere(dev, mxfp4_dequantize_nhwc, q, dtype)
    out = _empty(rows, cols, dtype=dtype, device=dev)
    rc = _lib.mxfp4_dequantize(codes.data_ptr(), scales.data_ptr(), rows, cols, d, out.data_ptr(),
                               _stream(dev.index))
    if rc:
        _fail("mxfp4_dequantize", rc)
    return out


def mxfp4_linear_nhwc(x, w, bias=None, out_dtype=None, stream=None):
    """out[..., n] = sum_k Q(x)[..., k] * w[n, k] + bias[n], a 1x1 convolution on
    4-bit operands.

    x: [..., K] dense (quantised by the call) or an ``Mxfp4Tensor`` of K
    columns; w: an ``Mxfp4Tensor`` of N rows and K columns; bias: float32 [N] or
    None.  out: contiguous, in ``out_dtype`` (default: x's dtype, bfloat16 for packed x).
    """
    if _torch is None:
        _setup()
    if stream is not None:
        return _on(stream, w[0], mxfp4_linear_nhwc, x, w, bias, out_dtype)
    r = _fast.linear(x, w, bias, out_dtype)
    if r is not None:
        return r
    _check_packed(w, "w")
    codes, scales, N, wk = w
    dev = codes.device
    if _device() != dev.index:
        return _elsewhere(dev, mxfp4_linear_nhwc, x, w, bias, out_dtype)
    if isinstance(x, Mxfp4Tensor):
        _check_packed(x, "x")
        xc, xs, M, K = x
        _same_device(dev, xc, "x")
        if out_dtype is None:
            out_dtype = _torch.bfloat16
        ld, xd, xp, sp, shape = K, CONVIMG_MXFP4, xc.data_ptr(), xs.data_ptr(), (M, N)
    else:
        M, K, ld = _rows_of(x, "x")
        _same_device(dev, x, "x")
        xd, xp, sp, shape = _dtype(x.dtype, "x"), x.data_ptr(), None, (*x.shape[:-1], N)
        if out_dtype is None:
            out_dtype = x.dtype
    if K != wk:
        raise ValueError("x has %d columns, w %d" % (K, wk))
    od = _dtype(out_dtype, "out_dtype")
    b = _param(bias, N, dev, "bias")
    need = _linear_bytes(M, N, K, xd)
    out = _empty(*shape, dtype=out_dtype, device=dev)
    ws = _empty(need, dtype=_u8, device=dev) if need else None
    rc = _lib.mxfp4_linear_fwd(xp, ld, sp, xd, codes.data_ptr(), scales.data_ptr(), b, M, N, K, od, out.data_ptr(),
                               ws.data_ptr() if need else None, need, _stream(dev.index))
    if rc:
        _fail("mxfp4_linear_fwd", rc)
    return out


def mxfp4_linear_bwd_nhwc(dy, x, w, dx_dtype=None, stream=None):
    """(dx, dw, db): gradients of the linear layer on 4-bit operands.

    dy: [..., N]; x: [..., K] and w: [N, K], the forward input and weights
    before quantisation, of one dtype; x may also be the input kept in 8 bits,
    an ``Mxint8Tensor`` of K columns and dy's rows.  dx: x's shape (dy's
    without N, and K) in ``dx_dtype`` (default: w's dtype); dw: float32 [N, K];
    db: float32 [N].
    """
    if _torch is None:
        _setup()
    if stream is not None:
        return _on(stream, dy, mxfp4_linear_bwd_nhwc, dy, x, w, dx_dtype)
    r = _fast.linear_bwd(dy, x, w, dx_dtype)
    if r is not None:
        return r
    M, N, ldy = _rows_of(dy, "dy")
    dev = dy.device
    kept = isinstance(x, Mxint8Tensor)
    if kept:
        _check_kept(x, "x")
        mx, K, ldx = x.rows, x.cols, x.cols
        xp, xs, shape = x.codes.data_ptr(), x.scales.data_ptr(), dy.shape[:-1]
        _same_device(dev, x.codes, "x")
    else:
        mx, K, ldx = _rows_of(x, "x")
        xp, xs, shape = x.data_ptr(), None, x.shape[:-1]
        _same_device(dev, x, "x")
    if w.dim() != 2 or mx != M or dy.shape[:-1] != shape or w.shape != (N, K):
        raise ValueError("dy must be [..., N], x [..., K] and w [N, K]")
    if not kept and x.dtype != w.dtype:
        raise TypeError("x and w must have one dtype")
    ldw = _rows_of(w, "w")[2]
    _same_device(dev, w, "w")
    if _device() != dev.index:
        return _elsewhere(dev, mxfp4_linear_bwd_nhwc, dy, x, w, dx_dtype)
    if dx_dtype is None:
        dx_dtype = w.dtype
    dd, wd, od = _dtype(dy.dtype, "dy"), _dtype(w.dtype, "w"), _dtype(dx_dtype, "dx_dtype")
    need = _linear_bwd_bytes(M, N, K)
    dx = _empty(*shape, K, dtype=dx_dtype, device=dev)
    dw, db = _empty(N, K, dtype=_f32, device=dev), _empty(N, dtype=_f32, device=dev)
    ws = _empty(need, dtype=_u8, device=dev)
    rest = (w.data_ptr(), ldw, wd, M, N, K, od, dx.data_ptr(), dw.data_ptr(), db.data_ptr(), ws.data_ptr(), need,
            _stream(dev.index))
    if kept:
        rc = _lib.mxfp4_linear_bwd_mxint8(dy.data_ptr(), ldy, dd, xp, xs, *rest)
    else:
        rc = _lib.mxfp4_linear_bwd(dy.data_ptr(), ldy, dd, xp, ldx, *rest)
    if rc:
        _fail("mxfp4_linear_bwd", rc)
    return dx, dw, db


# ---- activations kept in 8 bits -------------------------------------------

def _kept(device, rows, cols):
    return Mxint8Tensor(_empty(rows, -(-cols // 32) * 32, dtype=_i8, device=device),
                        _empty(rows, -(-cols // 128) * 4, dtype=_u8, device=device), rows, cols)


def _check_kept(q, what):
    codes, scales, rows, cols = q
    if not codes.is_cuda or codes.device != scales.device or codes.dtype is not _i8 or scales.dtype is not _u8 \
            or codes.shape != (rows, -(-cols // 32) * 32) or scales.shape != (rows, -(-cols // 128) * 4) \
            or cols <= 0 or not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError("%s is not an 8-bit operand of %d rows and %d columns" % (what, rows, cols))
    _fits(rows, cols, what)


def mxint8_quantize_nhwc(x, stream=None):
    """x [..., C] kept in 8 bits: an ``Mxint8Tensor``, a little over half of bfloat16's size."""
    if _torch is None:
        _setup()
    if stream is not None:
        return _on(stream, x, mxint8_quantize_nhwc, x)
    r = _fast.quantize8(x)
    if r is not None:
        return _new(Mxint8Tensor, r)
    rows, cols, ld = _rows_of(x, "x")
    dev = x.device
    if _device() != dev.index:
        return _elsewhere(dev, mxint8_quantize_nhwc, x)
    xd = _dtype(x.dtype, "x")
    q = _kept(dev, rows, cols)
    rc = _lib.mxint8_quantize(x.data_ptr(), ld, rows, cols, xd, q.codes.data_ptr(), q.scales.data_ptr(),
                              _stream(dev.index))
    if rc:
        _fail("mxint8_quantize", rc)
    return q


def mxint8_dequantize_nhwc(q, dtype, stream=None):
    """The values [rows, cols] that 8-bit rows stand for, in ``dtype`` (exact in bfloat16 and float32)."""
    if _torch is None:
        _setup()
    if stream is not None:
        return _on(stream, q[0], mxint8_dequantize_nhwc, q, dtype)
    r = _fast.dequantize8(q, dtype)
    if r is not None:
        return r
    _check_kept(q, "q")
    d = _dtype(dtype, "dtype")
    codes, scales, rows, cols = q
    dev = codes.device
    if _device() != dev.index:
        return _elsewhere(dev, mxint8_dequantize_nhwc, q, dtype)
    out = _empty(rows, cols, dtype=dtype, device=dev)
    rc = _lib.mxint8_dequantize(codes.data_ptr(), scales.data_ptr(), rows, cols, d, out.data_ptr(), _stream(dev.index))
    if rc:
        _fail("mxint8_dequantize", rc)
    return out


def layer_norm_mxint8_nhwc(x, gamma=None, beta=None, eps=1e-5, out_dtype=None, stream=None):
    """layer_norm_nhwc for training with what its gradient needs in 8 bits.

    Returns (y, kept, rstd): y as ``layer_norm_nhwc`` gives it, kept the
    normalised rows (x - mean) / sqrt(var + eps) as an ``Mxint8Tensor`` and rstd
    float32 of x's shape without the last dimension, for
    ``layer_norm_bwd_mxint8_nhwc``; neither x nor the mean is needed there.
    """
    if _torch is None:
        _setup()
    if stream is not None:
        return _on(stream, x, layer_norm_mxint8_nhwc, x, gamma, beta, eps, out_dtype)
    r = _fast.layer_norm_kept(x, gamma, beta, eps, out_dtype)
    if r is not None:
        return r[0], _new(Mxint8Tensor, r[1]), r[2]
    rows, cols, ld = _rows_of(x, "x")
    dev = x.device
    if _device() != dev.index:
        return _elsewhere(dev, layer_norm_mxint8_nhwc, x, gamma, beta, eps, out_dtype)
    if out_dtype is None:
        out_dtype = x.dtype
    xd, yd = _dtype(x.dtype, "x"), _dtype(out_dtype, "out_dtype")
    g, b = _param(gamma, cols, dev, "gamma"), _param(beta, cols, dev, "beta")
    y, q = _like(x, out_dtype), _kept(dev, rows, cols)
    rstd = _empty(x.shape[:-1], dtype=_f32, device=dev)
    rc = _lib.layer_norm_fwd_mxint8(x.data_ptr(), ld, g, b, rows, cols, eps, xd, yd, y.data_ptr(), q.codes.data_ptr(),
                                    q.scales.data_ptr(), rstd.data_ptr(), _stream(dev.index))
    if rc:
        _fail("layer_norm_fwd_mxint8", rc)
    return y, q, rstd


def layer_norm_bwd_mxint8_nhwc(dy, kept, gamma, rstd, dx_dtype=None, stream=None):
    """(dx, dgamma, dbeta): gradients of layer_norm_mxint8_nhwc.

    dy: [..., C] bfloat16, float16 or float32; kept, rstd: what the forward
    call returned; gamma: float32 [C] or None.  dx: contiguous, of dy's shape in
    ``dx_dtype`` (default: dy's dtype); dgamma and dbeta: float32 [C].
    """
    if _torch is None:
        _setup()
    if stream is not None:
        return _on(stream, dy, layer_norm_bwd_mxint8_nhwc, dy, kept, gamma, rstd, dx_dtype)
    r = _fast.layer_norm_kept_bwd(dy, kept, gamma, rstd, dx_dtype)
    if r is not None:
        return r
    rows, cols, ldy = _rows_of(dy, "dy")
    dev = dy.device
    _check_kept(kept, "kept")
    _same_device(dev, kept.codes, "kept")
    if (kept.rows, kept.cols) != (rows, cols):
        raise ValueError("dy has %d rows of %d columns, kept %d of %d" % (rows, cols, kept.rows, kept.cols))
    if _device() != dev.index:
        return _elsewhere(dev, layer_norm_bwd_mxint8_nhwc, dy, kept, gamma, rstd, dx_dtype)
    if dx_dtype is None:
        dx_dtype = dy.dtype
    dd, od = _dtype(dy.dtype, "dy"), _dtype(dx_dtype, "dx_dtype")
    g = _param(gamma, cols, dev, "gamma")
    rstd = rstd.reshape(-1).contiguous()      # (held until the call is made: it may be a copy)
    r = _param(rstd, rows, dev, "rstd")
    need = _norm_bwd_bytes(rows, cols)
    dx = _like(dy, dx_dtype)
    dgamma, dbeta = _empty(cols, dtype=_f32, device=dev), _empty(cols, dtype=_f32, device=dev)
    ws = _empty(need, dtype=_u8, device=dev)
    rc = _lib.layer_norm_bwd_mxint8(dy.data_ptr(), ldy, kept.codes.data_ptr(), kept.scales.data_ptr(), g, r, rows, cols,
                                    dd, od, dx.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr(), ws.data_ptr(), need,
                                    _stream(dev.index))
    if rc:
        _fail("layer_norm_bwd_mxint8", rc)
    return dx, dgamma, dbeta


# ---- low-rank adapters beside the linear layer ----------------------------

def _check_adapters(adapters, dev, N, K):
    """(number, rank, dtype code) of the adapters of a layer K -> N."""
    down, up, scale = adapters
    if down.dim() != 3 or up.dim() != 3 or not down.shape[0] or not down.shape[1] \
            or down.shape != (up.shape[0], up.shape[1], K) or up.shape[2] != N:
        raise ValueError("the adapters of a layer %d -> %d must be down [G, r, %d] and up [G, r, %d]" % (K, N, K, N))
    if not down.is_contiguous() or not up.is_contiguous():
        raise ValueError("the adapters must be contiguous")
    if down.dtype != up.dtype:
        raise TypeError("down and up must have one dtype")
    _same_device(dev, down, "down")
    _same_device(dev, up, "up")
    G, r = down.shape[:2]
    _fits(G, r, "down")
    if scale is None:
        raise ValueError("scale must be a contiguous float32 tensor of %d values on the input's device" % G)
    _param(scale, G, dev, "scale")
    return G, r, _dtype(down.dtype, "down")


def _check_ids(ids, shape, dev):
    if ids.dtype is not _i32 or ids.shape != shape or ids.device != dev or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 tensor of the rows' shape on the input's device")


def mxfp4_linear_adapters_nhwc(x, w, bias, adapters, ids, out_dtype=None, save=False, stream=None):
    """The linear layer of mxfp4_linear_nhwc with a low-rank adapter a row:

        out[...] = Q(x) w^T + bias + scale[g] * (x down[g]^T) up[g],  g = ids[...]

    x: [..., K] dense; w: an ``Mxfp4Tensor`` of N rows and K columns; bias:
    float32 [N] or None; adapters: ``Adapters``; ids: int32 of x's shape without
    the last dimension, in any order, a number outside 0 .. G-1 for a row
    without adapter.  out: contiguous [..., N] in ``out_dtype`` (default: x's
    dtype).  With ``save`` (out, kept, h) for mxfp4_linear_adapters_bwd_nhwc:
    x as an ``Mxint8Tensor`` and x down[g]^T, float32 [..., r] (0 without
    adapter).
    """
    if _torch is None:
        _setup()
    if stream is not None:
        return _on(stream, x, mxfp4_linear_adapters_nhwc, x, w, bias, adapters, ids, out_dtype, save)
    r = _fast.adapters(x, w, bias, adapters, ids, out_dtype, save)
    if r is not None:
        return (r[0], _new(Mxint8Tensor, r[1]), r[2]) if save else r
    M, K, ld = _rows_of(x, "x")
    dev = x.device
    _check_packed(w, "w")
    codes, scales, N, wk = w
    _same_device(dev, codes, "w")
    if K != wk:
        raise ValueError("x has %d columns, w %d" % (K, wk))
    G, rank, ad = _check_adapters(adapters, dev, N, K)
    _check_ids(ids, x.shape[:-1], dev)
    if _device() != dev.index:
        return _elsewhere(dev, mxfp4_linear_adapters_nhwc, x, w, bias, adapters, ids, out_dtype, save)
    if out_dtype is None:
        out_dtype = x.dtype
    xd, od = _dtype(x.dtype, "x"), _dtype(out_dtype, "out_dtype")
    b = _param(bias, N, dev, "bias")
    need = _adapters_bytes(M, N, K, G, rank, xd)
    out = _empty(*x.shape[:-1], N, dtype=out_dtype, device=dev)
    kept = _kept(dev, M, K) if save else None
    h = _empty(*x.shape[:-1], rank, dtype=_f32, device=dev) if save else None
    ws = _empty(need, dtype=_u8, device=dev)
    down, up, scale = adapters
    rc = _lib.mxfp4_linear_adapters_fwd(x.data_ptr(), ld, xd, codes.data_ptr(), scales.data_ptr(), b, down.data_ptr(),
                                        up.data_ptr(), scale.data_ptr(), ids.data_ptr(), G, rank, ad, M, N, K, od,
                                        out.data_ptr(), h.data_ptr() if save else None,
                                        kept.codes.data_ptr() if save else None,
                                        kept.scales.data_ptr() if save else None, ws.data_ptr(), need,
                                        _stream(dev.index))
    if rc:
        _fail("mxfp4_linear_adapters_fwd", rc)
    return (out, kept, h) if save else out


def mxfp4_linear_adapters_bwd_nhwc(dy, x, wt, adapters, ids, h, dx_dtype=None, stream=None):
    """(dx, ddown, dup): gradients of mxfp4_linear_adapters_nhwc, w and bias
    frozen.

    dy: [..., N]; x: the forward input, [..., K] or kept as an ``Mxint8Tensor``;
    wt: w's transpose quantised along N, an ``Mxfp4Tensor`` of K rows and N
    columns (``mxfp4_quantize_nhwc(w, transpose=True)``), or None to skip dx
    (then None is returned for it); adapters, ids: the forward call's; h: what
    it returned, float32 [..., r].  dx: [..., K] in ``dx_dtype`` (default: dy's
    dtype); ddown, dup: float32 of down's and up's shapes.
    """
    if _torch is None:
        _setup()
    if stream is not None:
        return _on(stream, dy, mxfp4_linear_adapters_bwd_nhwc, dy, x, wt, adapters, ids, h, dx_dtype)
    r = _fast.adapters_bwd(dy, x, wt, adapters, ids, h, dx_dtype)
    if r is not None:
        return r
    M, N, ldy = _rows_of(dy, "dy")
    dev = dy.device
    if isinstance(x, Mxint8Tensor):
        _check_kept(x, "x")
        _same_device(dev, x.codes, "x")
        mx, K, ldx, shape = x.rows, x.cols, x.cols, dy.shape[:-1]
        xd, xp, xs = CONVIMG_MXINT8, x.codes.data_ptr(), x.scales.data_ptr()
    else:
        mx, K, ldx = _rows_of(x, "x")
        _same_device(dev, x, "x")
        xd, xp, xs, shape = _dtype(x.dtype, "x"), x.data_ptr(), None, x.shape[:-1]
    if mx != M or dy.shape[:-1] != shape:
        raise ValueError("dy must be [..., N] and x [..., K] of the same rows")
    if wt is not None:
        _check_packed(wt, "wt")
        _same_device(dev, wt[0], "wt")
        if wt[2:] != (K, N):
            raise ValueError("wt has %d rows of %d columns; K is %d and N %d" % (*wt[2:], K, N))
    G, rank, ad = _check_adapters(adapters, dev, N, K)
    _check_ids(ids, dy.shape[:-1], dev)
    if h.dtype is not _f32 or h.device != dev or h.shape != (*dy.shape[:-1], rank) or not h.is_contiguous():
        raise ValueError("h must be a contiguous float32 tensor [..., %d] on the input's device" % rank)
    if _device() != dev.index:
        return _elsewhere(dev, mxfp4_linear_adapters_bwd_nhwc, dy, x, wt, adapters, ids, h, dx_dtype)
    if dx_dtype is None:
        dx_dtype = dy.dtype
    dd, od = _dtype(dy.dtype, "dy"), _dtype(dx_dtype, "dx_dtype")
    need = _adapters_bwd_bytes(M, N, K, G, rank)
    dx = None if wt is None else _empty(*dy.shape[:-1], K, dtype=dx_dtype, device=dev)
    down, up, scale = adapters
    ddown, dup = _empty(G, rank, K, dtype=_f32, device=dev), _empty(G, rank, N, dtype=_f32, device=dev)
    ws = _empty(need, dtype=_u8, device=dev)
    rc = _lib.mxfp4_linear_adapters_bwd(dy.data_ptr(), ldy, dd, xp, ldx, xs, xd,
                                        None if wt is None else wt[0].data_ptr(),
                                        None if wt is None else wt[1].data_ptr(), down.data_ptr(), up.data_ptr(),
                                        scale.data_ptr(), ids.data_ptr(), G, rank, ad, h.data_ptr(), M, N, K, od,
                                        None if wt is None else dx.data_ptr(), ddown.data_ptr(), dup.data_ptr(),
                                        ws.data_ptr(), need, _stream(dev.index))
    if rc:
        _fail("mxfp4_linear_adapters_bwd", rc)
    return dx, ddown, dup
