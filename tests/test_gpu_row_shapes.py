"""Sizes at which the row operators change their kernels, operands beyond 32-bit offsets, and vectors, against the
definitions in 64 bits (row_reference.py has them and the tolerances)."""
import numpy as np
import pytest
import torch

import convolution_implicit_gemm_fwd_amd as cim
import row_reference as ref
from gpu_harness import need_gpu
from row_reference import f64
from test_gpu_layer_norm import EPS, check_bwd, params, stats_of
from test_gpu_layer_norm import rows as norm_rows
from test_gpu_mxfp4 import check_bwd as check_linear_bwd
from test_gpu_mxfp4 import check_linear, rows, same_packed

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


# tiles of 256, of 128, 128 x 64 with two groups of waves, 64, 64 x 32 and 32 with four groups; K that fills the last
# K tile, ends inside it, inside a scale dword, or leaves the last groups nothing
@pytest.mark.parametrize("M,N,K", [(3100, 3100, 1030), (4200, 4150, 300), (3100, 3100, 256), (3073, 3201, 130), (1800, 1700, 288),
                                   (1667, 2000, 1000), (500, 4099, 1056),
                                   (1000, 1600, 1250), (900, 900, 513), (129, 6500, 2050), (65, 4100, 1100), (40, 8100, 1030),
                                   (33, 300, 4127), (7, 50, 1057), (256, 129, 8200), (5, 33, 33000)])
def test_linear_shapes(M, N, K):
    check_linear(M, N, K, BF16, FP32)
    check_linear(M, N, K, FP16, BF16, bias=False, packed=True)


# rows that the product quantises itself: up to 4 rows and 32768 values
@pytest.mark.parametrize("M,K", [(1, 1), (1, 31), (1, 256), (1, 300), (1, 4096), (1, 6200), (1, 32768), (1, 32769), (2, 5000),
                                 (2, 16384), (2, 16385), (3, 100), (3, 10922), (4, 129), (4, 2048), (4, 8192), (4, 8193), (5, 64)])
@pytest.mark.parametrize("xt,out", [(BF16, BF16), (FP32, FP16), (FP16, FP32)])
def test_few_rows(M, K, xt, out):
    for N, pad, offset in ((16, 0, 0), (77, 3, 1)):
        check_linear(M, N, K, xt, out, pad=pad, offset=offset)
    check_linear(M, 5, K, xt, out, bias=False)


def test_few_rows_keep_a_nan_to_its_row():
    x = rows(1, 4, 700, FP32)
    w = cim.mxfp4_quantize_nhwc(rows(2, 100, 700, FP32))
    clean = cim.mxfp4_linear_nhwc(x, w)
    x[1, 699], x[2, 0] = float("nan"), float("-inf")
    y = cim.mxfp4_linear_nhwc(x, w)
    assert torch.isnan(y[1:3]).all() and torch.equal(y[0::3], clean[0::3])


def test_weights_with_a_nan_block_reach_their_column_only():
    for M in (2, 40, 300):
        x, v = rows(1, M, 300, BF16), rows(2, 200, 300, FP32)
        clean = cim.mxfp4_linear_nhwc(x, cim.mxfp4_quantize_nhwc(v))
        v[7, 299] = float("inf")
        y = cim.mxfp4_linear_nhwc(x, cim.mxfp4_quantize_nhwc(v))
        assert torch.isnan(y[:, 7]).all()
        keep = [n for n in range(200) if n != 7]
        assert torch.equal(y[:, keep], clean[:, keep])


# products of like and of unlike size, tiles of each edge, parts of 128 rows
@pytest.mark.parametrize("M,N,K", [(3000, 2900, 200), (64, 2200, 2300), (3000, 70, 60), (127, 128, 129), (130, 1500, 1400),
                                   (2, 300, 700), (1500, 260, 2000)])
def test_linear_backward_shapes(M, N, K):
    check_linear_bwd(M, N, K, BF16, BF16, FP32)
    check_linear_bwd(M, N, K, FP32, FP16, BF16, pad=5, offset=1)


@pytest.mark.parametrize("n,cols", [(140000, 24), (70000, 40), (3, 8193), (2, 12000), (70, 8192), (600, 5000), (4, 4096),
                                    (5, 4096), (2600, 1536), (40, 33)])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (FP32, FP16)])
def test_layer_norm_walks_rows(n, cols, dtype, out):
    """More rows than one pass of the resident workgroups, one pass exactly, and the bounds between kernels."""
    x = norm_rows(n, n, cols, dtype, mean=2.0)
    g, b = params(cols, cols)
    got, mean, rstd = cim.layer_norm_nhwc(x, g, b, EPS, out_dtype=out, stats=True)
    y, m, r, dy, dm, dr = ref.layer_norm(f64(x), f64(g), f64(b), EPS, out)
    ref.check(got, y, dy, "y")
    ref.check(mean, m, dm, "mean")
    ref.check(rstd, r, dr, "rstd")
    check_bwd(x, norm_rows(n + 1, n, cols, out, scale=0.1, mean=0), g, dtype)


def test_vectors():
    """A single row without a row dimension."""
    x, g = norm_rows(1, 1, 200, BF16)[0], params(1, 200)[0]
    y, mean, rstd = cim.layer_norm_nhwc(x, g, None, EPS, stats=True)
    assert y.shape == (200,) and mean.shape == () and rstd.shape == ()
    want, _, _, tol, _, _ = ref.layer_norm(f64(x)[None], f64(g), None, EPS, BF16)
    ref.check(y[None], want, tol, "vector")
    dx, dg, db = cim.layer_norm_bwd_nhwc(y, x, g, mean, rstd)
    assert dx.shape == (200,) and dg.shape == (200,)
    w = cim.mxfp4_quantize_nhwc(rows(2, 30, 200, FP32))
    assert torch.equal(cim.mxfp4_linear_nhwc(x, w), cim.mxfp4_linear_nhwc(x[None], w)[0])
    assert cim.mxfp4_quantize_nhwc(x, transpose=True).codes.shape == (200, 16)


def far_rows(seed, n, cols, dtype, ld):
    """n rows of which the last starts beyond 2^32 bytes."""
    flat = torch.empty((n - 1) * ld + cols, dtype=dtype, device="cuda")
    t = torch.as_strided(flat, (n, cols), (ld, 1))
    t.copy_(rows(seed, n, cols, dtype))
    return t


def test_offsets_beyond_32_bits():
    n, cols, ld = 5, 300, (1 << 29) + 7          # 4 GiB + from the first row to the last, in 2-byte elements
    x, dy = far_rows(1, n, cols, BF16, ld), far_rows(2, n, cols, BF16, ld)
    y, _, _, tol, _, _ = ref.layer_norm(f64(x), None, None, EPS, FP32)
    ref.check(cim.layer_norm_nhwc(x, out_dtype=FP32), y, tol, "layer norm")
    check_bwd(x, dy, None, FP32)
    for transpose in (False, True):
        same_packed(cim.mxfp4_quantize_nhwc(x, transpose=transpose), f64(x).T if transpose else f64(x))
    w = rows(3, 40, cols, FP32)
    q = cim.mxfp4_quantize_nhwc(w)
    for m in (3, 5):
        got = cim.mxfp4_linear_nhwc(x[n - m:], q, out_dtype=FP32)
        want, tol = ref.product(ref.mx_quantize(f64(x[n - m:]))[2], ref.mx_quantize(f64(w))[2], None, FP32)
        ref.check(got, want, tol, "linear")
    dx, dw, db = cim.mxfp4_linear_bwd_nhwc(rows(4, n, 40, BF16), x, rows(5, 40, cols, BF16))
    near = cim.mxfp4_linear_bwd_nhwc(rows(4, n, 40, BF16), x.contiguous(), rows(5, 40, cols, BF16))
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), near))


def test_backward_repeats_bit_for_bit():
    dy, x, w = rows(1, 3000, 200, BF16), rows(2, 3000, 300, BF16), rows(3, 200, 300, BF16)
    first = cim.mxfp4_linear_bwd_nhwc(dy, x, w)
    mean, rstd = stats_of(x)
    norm = cim.layer_norm_bwd_nhwc(x, x, None, mean, rstd)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, cim.mxfp4_linear_bwd_nhwc(dy, x, w)))
        assert all(torch.equal(a, b) for a, b in zip(norm, cim.layer_norm_bwd_nhwc(x, x, None, mean, rstd)))
