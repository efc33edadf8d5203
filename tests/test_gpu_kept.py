"""Activations kept in 8 bits on the GPU: rows, layer norm with its gradient
and the linear layer's gradient, against the definitions in 64 bits
(kept_reference.py has them and the tolerances)."""
import numpy as np
import pytest
import torch

import convolution_implicit_gemm_fwd_amd as cim
import kept_reference as kept
import row_reference as ref
from gpu_harness import need_gpu
from row_reference import f64
from test_gpu_layer_norm import params
from test_gpu_layer_norm import rows as norm_rows
from test_gpu_mxfp4 import rows

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5
SIZES = [(1, 1), (1, 32), (3, 33), (40, 64), (7, 100), (33, 129), (5, 511), (130, 640), (64, 1000), (2, 4096), (1, 9000),
         (513, 96), (300, 300)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def same(q, x64):
    codes, scales, val, bad = kept.quantize(x64)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    got = q.codes.cpu().numpy().reshape(codes.shape[0], -1, 32)
    assert np.array_equal(got[~bad], codes.reshape(got.shape)[~bad])
    return val


@pytest.mark.parametrize("n,cols", SIZES)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
def test_rows(n, cols, dtype, pad, offset):
    x = rows(n + cols, n, cols, dtype, pad, offset)
    q = cim.mxint8_quantize_nhwc(x)
    val = same(q, f64(x))
    assert np.abs(val - f64(x)).max() <= np.ldexp(0.5, int(q.scales.max()) - 127)
    for out in (BF16, FP32):      # exact
        assert np.array_equal(f64(cim.mxint8_dequantize_nhwc(q, out)), val)
    want = torch.from_numpy(val).to(FP16).double().numpy()
    assert np.array_equal(f64(cim.mxint8_dequantize_nhwc(q, FP16)), want)


def test_every_rounding():
    """Every code and tie and the values beside, with the unit fixed by the first value; both sides of the unit's step;
    zeros; the largest and smallest numbers."""
    k = np.arange(-127, 128)
    for scale in (1.0, 2.0 ** -126, 2.0 ** -60, 2.0 ** 120):
        marks = np.unique(np.concatenate([k, k + 0.5, k + 0.5 - 2.0 ** -10, k + 0.5 + 2.0 ** -10]))
        marks = marks[np.abs(marks) <= 127]
        n = -(-len(marks) // 31)
        x = np.zeros((n, 31))
        x.reshape(-1)[:len(marks)] = marks
        x = np.concatenate([np.full((n, 1), 127.0), x], 1) * scale
        same(cim.mxint8_quantize_nhwc(torch.from_numpy(x).float().cuda()), x)
    top = np.float32([127, np.nextafter(np.float32(127), np.float32(128)), 127.5, 128, 64, 63.5, 63.50001, 1, 0])
    x = np.zeros((len(top) * 3, 32), np.float32)
    for i, f in enumerate((1.0, 2.0 ** 121, 2.0 ** -130)):
        x[i * len(top):(i + 1) * len(top), 5] = (top.astype(np.float64) * f).astype(np.float32)
    x[0, 7] = -1.5
    same(cim.mxint8_quantize_nhwc(torch.from_numpy(x).cuda()), x.astype(np.float64))
    big = torch.full((2, 40), torch.finfo(FP32).max, device="cuda")
    same(cim.mxint8_quantize_nhwc(big), f64(big))
    small = torch.full((2, 40), 2.0 ** -149, device="cuda")
    same(cim.mxint8_quantize_nhwc(small), f64(small))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_infinities_stay_in_their_block(dtype):
    x = rows(1, 6, 200, dtype)
    x[1, 40] = float("nan")
    x[2, 199] = float("inf")
    x[4, 0] = float("-inf")
    q = cim.mxint8_quantize_nhwc(x)
    val = same(q, f64(x))
    got = f64(cim.mxint8_dequantize_nhwc(q, FP32))
    assert np.array_equal(np.isnan(got), np.isnan(val)) and np.isnan(got).sum() == 32 + 8 + 32


def test_maps_and_no_rows():
    x = rows(2, 24, 40, BF16).view(2, 3, 4, 40)
    q = cim.mxint8_quantize_nhwc(x)
    assert (q.rows, q.cols) == (24, 40)
    same(q, f64(x).reshape(24, 40))
    q = cim.mxint8_quantize_nhwc(x[:0])
    assert q.rows == 0 and cim.mxint8_dequantize_nhwc(q, FP32).shape == (0, 40)


NORM = [(1, 1), (1, 7), (3, 8), (5, 31), (2, 32), (65, 33), (130, 64), (17, 100), (9, 128), (7, 250), (33, 256), (4, 511),
        (6, 513), (3, 1000), (2, 1024), (5, 2013), (3, 2048), (1, 4096), (2, 4097), (3, 6000), (2, 8192), (1, 10001),
        (2, 16391)]


@pytest.mark.parametrize("n,cols", NORM)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (FP32, FP32), (FP16, BF16)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (5, 3)])
def test_norm(n, cols, dtype, out, pad, offset):
    x = norm_rows(cols, n, cols, dtype, pad, offset)
    g, b = params(cols, cols)
    for gg, bb in ((g, b), (None, b), (g, None)):
        y, q, rstd = cim.layer_norm_mxint8_nhwc(x, gg, bb, EPS, out_dtype=out)
        want, _, r, dy, _, dr = ref.layer_norm(f64(x), None if gg is None else f64(gg), None if bb is None else f64(bb),
                                               EPS, out)
        ref.check(y, want, dy, "y")
        ref.check(rstd, r, dr, "rstd")
        nn, _, dn, _ = kept.norm(f64(x), EPS)
        kept.check_kept(q, nn, dn, "kept")


def test_norm_hard_rows():
    """A constant row keeps zeros; a mean far above the spread; an infinity or a NaN stays in its row."""
    x = norm_rows(4, 6, 96, FP32)
    x[0] = 3.0
    x[1] = 1e4 + x[1]
    x[3, 5] = float("inf")
    x[4, 95] = float("nan")
    y, q, rstd = cim.layer_norm_mxint8_nhwc(x, None, None, EPS)
    assert not q.codes[0].any() and not y[0].any()
    assert (q.scales[3:5, :3] == 255).all() and not torch.isfinite(y[3:5]).any()
    fine = [1, 2, 5]
    n, _, dn, _ = kept.norm(f64(x[fine]), EPS)
    kept.check_kept(cim.Mxint8Tensor(q.codes[fine], q.scales[fine], 3, 96), n, dn, "kept")


@pytest.mark.parametrize("n,cols", NORM + [(700, 64), (1500, 130), (300, 1500)])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (FP32, BF16), (FP16, FP32), (FP32, FP32)])
@pytest.mark.parametrize("pad", [0, 5])
def test_norm_gradient(n, cols, dtype, out, pad):
    dy = norm_rows(7 + cols, n, cols, dtype, pad, pad)
    q = cim.mxint8_quantize_nhwc(norm_rows(cols, n, cols, FP32, mean=0.0))
    rstd = torch.from_numpy(np.random.default_rng(5).uniform(0.5, 2, n).astype(np.float32)).cuda()
    g, _ = params(cols, cols)
    for gg in (g, None):
        dx, dg, db = cim.layer_norm_bwd_mxint8_nhwc(dy, q, gg, rstd, dx_dtype=out)
        w = kept.norm_bwd(f64(dy), kept.values(q), None if gg is None else f64(gg), f64(rstd), out)
        ref.check(dx, w[0], w[3], "dx")
        ref.check(dg, w[1], w[4], "dgamma")
        ref.check(db, w[2], w[5], "dbeta")


def test_norm_gradient_by_differences():
    """Against differences of the function that the kept rows belong to: sum(dy * y) by x, gamma and beta, where the
    kept rows are n to 8 bits (so to that precision)."""
    g = np.random.default_rng(3)
    x = g.standard_normal((4, 64))
    gamma, beta, dy = 1 + 0.2 * g.standard_normal(64), 0.1 * g.standard_normal(64), g.standard_normal((4, 64))

    def f(x, gamma, beta):
        n = (x - x.mean(-1, keepdims=True)) / np.sqrt(x.var(-1, keepdims=True) + EPS)
        return (dy * (n * gamma + beta)).sum()
    def cuda(a):
        return torch.from_numpy(a.astype(np.float32)).cuda()
    _, q, rstd = cim.layer_norm_mxint8_nhwc(cuda(x), cuda(gamma), cuda(beta), EPS)
    dx, dg, db = (f64(t) for t in cim.layer_norm_bwd_mxint8_nhwc(cuda(dy), q, cuda(gamma), rstd))
    # n is off by at most half a unit, 2^-6 where |n| < 4: dx = r (h - mean h - n mean(h n)) moves by r (dn |mean(h n)| +
    # |n| mean(|h|) dn), dgamma by the sum of |dy| dn
    dn, r, h = 2.0 ** -6, f64(rstd)[:, None], np.abs(dy * gamma)
    tol = r * dn * (np.abs((dy * gamma * f64(x_hat(x))).mean(-1, keepdims=True)) + np.abs(f64(x_hat(x))) * h.mean(-1, keepdims=True) + dn * h.mean(-1, keepdims=True)) + 1e-4
    step = 1e-5
    for k in range(0, 256, 7):
        e = np.zeros(256)
        e[k] = step
        d = (f(x + e.reshape(4, 64), gamma, beta) - f(x - e.reshape(4, 64), gamma, beta)) / (2 * step)
        assert abs(dx.reshape(-1)[k] - d) <= tol.reshape(-1)[k]
    for k in range(64):
        e = np.zeros(64)
        e[k] = step
        assert abs(dg[k] - (f(x, gamma + e, beta) - f(x, gamma - e, beta)) / (2 * step)) <= dn * np.abs(dy[:, k]).sum() + 1e-4
        assert abs(db[k] - (f(x, gamma, beta + e) - f(x, gamma, beta - e)) / (2 * step)) <= 1e-4


def x_hat(x):
    return torch.from_numpy((x - x.mean(-1, keepdims=True)) / np.sqrt(x.var(-1, keepdims=True) + EPS))


def test_norm_no_rows():
    x = norm_rows(5, 6, 48, FP32).view(2, 3, 48)[:0]
    y, q, rstd = cim.layer_norm_mxint8_nhwc(x)
    assert y.shape == x.shape and q.rows == 0 and rstd.shape == (0, 3)
    dx, dg, db = cim.layer_norm_bwd_mxint8_nhwc(x, q, None, rstd)
    assert dx.shape == x.shape and not dg.any() and not db.any()


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (5, 33, 40), (64, 64, 64), (100, 70, 130), (129, 200, 96), (300, 48, 257),
                                   (1000, 96, 33)])
@pytest.mark.parametrize("dtype,grad", [(BF16, BF16), (FP32, FP32), (FP16, FP32), (BF16, FP16)])
def test_linear_gradient(M, N, K, dtype, grad):
    dy, w = rows(1, M, N, grad, 2), rows(3, N, K, dtype, 1)
    q = cim.mxint8_quantize_nhwc(rows(2, M, K, FP32))
    dx, dw, db = cim.mxfp4_linear_bwd_nhwc(dy, q, w)
    a, x, ww = f64(dy), kept.values(q), f64(w)
    d = [ref.mx_quantize(t)[2] for t in (a, ww.T, a.T, x.T)]
    ref.check(dx, *ref.product(d[0], d[1], None, dtype), "dx")
    ref.check(dw, *ref.product(d[2], d[3], None, FP32), "dw")
    ref.check(db, a.sum(0), (M + 8) * ref.U * np.abs(a).sum(0) + 1e-40, "db")
    again = cim.mxfp4_linear_bwd_nhwc(dy, cim.mxint8_dequantize_nhwc(q, FP32), w.float()) if dtype == FP32 else None
    if again:      # the same operands from the values themselves
        assert all(torch.equal(p, r) for p, r in zip((dx, dw, db), again))


def test_linear_gradient_maps_and_no_rows():
    dy = rows(1, 24, 40, BF16).view(2, 3, 4, 40)
    w = rows(2, 40, 64, BF16)
    q = cim.mxint8_quantize_nhwc(rows(3, 24, 64, BF16).view(2, 3, 4, 64))
    dx, dw, db = cim.mxfp4_linear_bwd_nhwc(dy, q, w)
    assert dx.shape == (2, 3, 4, 64)
    flat = cim.mxfp4_linear_bwd_nhwc(dy.view(24, 40), q, w)
    assert torch.equal(dx.view(24, 64), flat[0]) and torch.equal(dw, flat[1]) and torch.equal(db, flat[2])
    q0 = cim.Mxint8Tensor(q.codes[:0], q.scales[:0], 0, 64)
    dx, dw, db = cim.mxfp4_linear_bwd_nhwc(dy[:0], q0, w)
    assert dx.shape == (0, 3, 4, 64) and not dw.any() and not db.any()
