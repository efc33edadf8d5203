"""Layer norm over channels and its gradient on the GPU, against the
definitions in 64 bits (row_reference.py has them and the tolerances)."""
import numpy as np
import pytest
import torch

import convolution_implicit_gemm_fwd_amd as cim
import row_reference as ref
from gpu_harness import need_gpu
from row_reference import f64

pytestmark = pytest.mark.gpu
EPS = 1e-5
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def rows(seed, n, cols, dtype, pad=0, offset=0, scale=1.0, mean=0.3):
    """[n, cols] on the device, `pad` columns to the next row, `offset` elements past an aligned start."""
    g = np.random.default_rng(seed)
    a = (g.standard_normal((n, cols + pad)) * scale + mean).astype(np.float32)
    t = torch.from_numpy(a).to(dtype)
    flat = torch.empty(t.numel() + offset, dtype=dtype, device="cuda")
    flat[offset:].copy_(t.reshape(-1))
    return flat[offset:].view(n, cols + pad)[:, :cols]


def params(seed, cols):
    g = np.random.default_rng(1000 + seed)
    return (torch.from_numpy((1 + 0.2 * g.standard_normal(cols)).astype(np.float32)).cuda(),
            torch.from_numpy((0.2 * g.standard_normal(cols)).astype(np.float32)).cuda())


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 31), (2, 32), (65, 33), (130, 64), (17, 100), (9, 128), (7, 250), (33, 256), (4, 511),
          (6, 513), (3, 1000), (2, 1024), (5, 2013), (3, 2048), (1, 4096), (2, 4097), (3, 6000), (2, 8192), (1, 10001),
          (2, 16384), (2, 16391), (1, 40000)]


@pytest.mark.parametrize("n,cols", SHAPES)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (FP32, BF16), (FP16, FP32)])
def test_forward(n, cols, dtype, out):
    x = rows(cols, n, cols, dtype)
    g, b = params(cols, cols)
    got, mean, rstd = cim.layer_norm_nhwc(x, g, b, EPS, out_dtype=out, stats=True)
    y, m, r, dy, dm, dr = ref.layer_norm(f64(x), f64(g), f64(b), EPS, out)
    ref.check(got, y, dy, "y")
    ref.check(mean, m, dm, "mean")
    ref.check(rstd, r, dr, "rstd")


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("out", [BF16, FP16, FP32])
@pytest.mark.parametrize("pad,offset", [(0, 0), (5, 3), (64, 1)])
def test_forward_types_and_strides(dtype, out, pad, offset):
    for n, cols in ((37, 200), (3, 1500)):
        x = rows(3, n, cols, dtype, pad, offset)
        g, b = params(3, cols)
        for gg, bb in ((g, b), (None, None), (g, None), (None, b)):
            y, _, _, tol, _, _ = ref.layer_norm(f64(x), None if gg is None else f64(gg), None if bb is None else f64(bb),
                                                EPS, out)
            ref.check(cim.layer_norm_nhwc(x, gg, bb, EPS, out_dtype=out), y, tol, "y")


def test_forward_map_and_empty():
    x = rows(5, 2 * 3 * 5, 48, FP32).view(2, 3, 5, 48)
    y = cim.layer_norm_nhwc(x, None, None, EPS)
    assert y.shape == x.shape
    want, _, _, tol, _, _ = ref.layer_norm(f64(x), None, None, EPS, FP32)
    ref.check(y, want, tol, "map")
    assert cim.layer_norm_nhwc(x[:0]).shape == (0, 3, 5, 48)
    dx, dg, db = cim.layer_norm_bwd_nhwc(x[:0], x[:0], None, x[:0, ..., 0], x[:0, ..., 0])
    assert dx.numel() == 0 and not dg.any() and not db.any()


def test_forward_hard_rows():
    """A constant row, a mean far above the spread, tiny and huge values; a NaN or an infinity stays in its row."""
    cols = 300
    g = np.random.default_rng(7)
    a = g.standard_normal((6, cols)).astype(np.float32)
    a[0] = 3.0
    a[1] = 4096 + a[1]
    a[2] *= 1e-18
    a[3] *= 1e15
    a[4] = 0
    x = torch.from_numpy(a).cuda()
    y, _, _, tol, _, _ = ref.layer_norm(f64(x), None, None, EPS, FP32)
    ref.check(cim.layer_norm_nhwc(x, eps=EPS), y, tol, "hard rows")
    x[2, 17], x[4, 299] = float("nan"), float("inf")
    z = cim.layer_norm_nhwc(x, eps=EPS)
    assert torch.isnan(z[2]).all() and torch.isnan(z[4]).all()
    keep = [0, 1, 3, 5]
    ref.check(z[keep], y[keep], tol[keep], "rows beside a NaN")


def stats_of(x):
    a = f64(x)
    m = a.mean(-1)
    r = 1 / np.sqrt(a.var(-1) + EPS)
    return torch.from_numpy(m.astype(np.float32)).cuda(), torch.from_numpy(r.astype(np.float32)).cuda()


def parts_chain(n):
    # rows a partial sum takes one after another, then the partial sums
    return -(-n // 256) + 256 + 16


def check_bwd(x, dy, g, out):
    mean, rstd = stats_of(x)
    dx, dg, db = cim.layer_norm_bwd_nhwc(dy, x, g, mean, rstd, dx_dtype=out)
    w = ref.layer_norm_bwd(f64(dy), f64(x), None if g is None else f64(g), f64(mean), f64(rstd), out,
                           parts_chain(x.shape[0]))
    ref.check(dx, w[0], w[3], "dx")
    ref.check(dg, w[1], w[4], "dgamma")
    ref.check(db, w[2], w[5], "dbeta")


@pytest.mark.parametrize("n,cols", SHAPES + [(700, 64), (3000, 16), (1030, 200), (600, 1024), (300, 4100)])
@pytest.mark.parametrize("dtype,grad,out", [(BF16, BF16, BF16), (FP32, BF16, FP16), (FP16, FP32, FP32)])
def test_backward(n, cols, dtype, grad, out):
    check_bwd(rows(cols, n, cols, dtype), rows(cols + 1, n, cols, grad, scale=0.1, mean=0), params(cols, cols)[0], out)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("grad", [BF16, FP16, FP32])
def test_backward_types_and_strides(dtype, grad):
    for n, cols, out in ((41, 200, BF16), (19, 1500, FP32)):
        for pad, offset in ((0, 0), (7, 1)):
            x, dy = rows(1, n, cols, dtype, pad, offset), rows(2, n, cols, grad, 2 * pad, offset, 0.1, 0)
            check_bwd(x, dy, params(3, cols)[0], out)
            check_bwd(x, dy, None, out)


def test_backward_against_differences():
    """Central differences of the forward definition in 64 bits, weighted by dy."""
    n, cols, h = 3, 40, 1e-5
    x, dy = rows(11, n, cols, FP32), rows(12, n, cols, FP32, mean=0)
    g, b = params(11, cols)
    mean, rstd = stats_of(x)
    dx, dg, db = (f64(t) for t in cim.layer_norm_bwd_nhwc(dy, x, g, mean, rstd))

    def loss(a, gg, bb):
        return (ref.layer_norm(a, gg, bb, EPS, FP32)[0] * f64(dy)).sum()

    a, gg, bb = f64(x), f64(g), f64(b)
    # the differences err by h^2 times a third derivative, and by 2^-53 of the loss over h
    for got, base, which in ((dx, a, 0), (dg, gg, 1), (db, bb, 2)):
        flat = base.reshape(-1)
        for k in range(0, flat.size, 7):
            e = np.zeros_like(flat)
            e[k] = h
            args = [[a, gg, bb], [a, gg, bb]]
            args[0][which], args[1][which] = (base + e.reshape(base.shape)), (base - e.reshape(base.shape))
            want = (loss(*args[0]) - loss(*args[1])) / (2 * h)
            assert abs(got.reshape(-1)[k] - want) <= 2e-5 * (1 + abs(want)), (which, k)


def test_backward_repeats_bit_for_bit():
    x, dy = rows(1, 5000, 96, BF16), rows(2, 5000, 96, BF16, mean=0)
    mean, rstd = stats_of(x)
    first = cim.layer_norm_bwd_nhwc(dy, x, None, mean, rstd)
    for _ in range(3):
        for p, q in zip(first, cim.layer_norm_bwd_nhwc(dy, x, None, mean, rstd)):
            assert torch.equal(p, q)


@pytest.mark.parametrize("n,cols", [(1, 1), (3, 32), (70, 64), (9, 100), (5, 513), (4, 1000), (2, 4096), (3, 4100), (2, 8200),
                                    (2, 17000)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_mxfp4_output_is_the_fp32_result_quantised(n, cols, dtype):
    x = rows(cols, n, cols, dtype, pad=3)
    g, b = params(cols, cols)
    q = cim.layer_norm_mxfp4_nhwc(x, g, b, EPS)
    y = cim.layer_norm_nhwc(x, g, b, EPS, out_dtype=FP32)
    codes, scales, _, _ = ref.mx_quantize(f64(y))
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
