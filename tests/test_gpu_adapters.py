"""Low-rank adapters of many requests beside the linear layer on the GPU,
against the definitions in 64 bits (kept_reference.py has them and the
tolerances)."""
import numpy as np
import pytest
import torch

import convolution_implicit_gemm_fwd_amd as cim
import kept_reference as kept
import row_reference as ref
from gpu_harness import need_gpu
from row_reference import U, f64
from test_gpu_mxfp4 import rows

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def layer(seed, N, K, G, r, dtype):
    g = np.random.default_rng(seed)
    def make(*shape):
        return torch.from_numpy((g.standard_normal(shape) / np.sqrt(shape[-2])).astype(np.float32)).to(dtype).cuda()
    w = rows(seed + 1, N, K, FP32)
    bias = torch.from_numpy(g.standard_normal(N).astype(np.float32)).cuda()
    scale = torch.from_numpy(g.uniform(0.25, 2, G).astype(np.float32)).cuda()
    return w, bias, cim.Adapters(make(G, r, K), make(G, r, N), scale)


def numbers(seed, M, G, order):
    """ids of M rows; some rows have none: -1, G or far outside."""
    g = np.random.default_rng(seed)
    ids = g.integers(0, G, M) if order == "mixed" else np.sort(g.integers(0, G, M))
    ids = np.where(g.random(M) < 0.15, g.choice([-1, G, 2 ** 31 - 1, -2 ** 31], M), ids)
    return torch.from_numpy(ids.astype(np.int32)).cuda()


def want_forward(x, w, bias, ad, ids, out):
    a, q = ref.mx_quantize(f64(x))[2], ref.mx_quantize(f64(w))[2]
    b = 0 if bias is None else f64(bias)
    mags = np.abs(a) @ np.abs(q).T + np.abs(b)
    return kept.beside(a @ q.T + b, (x.shape[1] / 32 + 40) * U * mags, mags, f64(x), f64(ad.down), f64(ad.up), f64(ad.scale),
                       f64(ids).astype(np.int64), out)


FORWARD = [(1, 1, 1, 1, 1), (1, 40, 33, 2, 5), (1, 300, 2500, 3, 16), (2, 64, 96, 1, 64), (3, 70, 513, 5, 17), (4, 130, 1000, 4, 70),
           (5, 33, 100, 3, 1), (17, 48, 640, 30, 8), (64, 96, 1024, 3, 16), (64, 520, 1200, 9, 33), (65, 100, 130, 4, 16),
           (130, 257, 300, 2, 40), (256, 96, 200, 6, 16), (257, 96, 200, 6, 16), (300, 64, 64, 7, 20), (400, 64, 264, 5, 130),
           (513, 140, 97, 1, 16), (700, 400, 160, 20, 130), (1700, 48, 520, 4, 24)]


@pytest.mark.parametrize("M,N,K,G,r", FORWARD)
@pytest.mark.parametrize("dtype,adtype,out", [(BF16, BF16, BF16), (FP32, FP32, FP32), (FP16, FP16, FP32), (FP16, BF16, FP16),
                                              (FP32, BF16, BF16)])
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_forward(M, N, K, G, r, dtype, adtype, out, order):
    x = rows(M + K, M, K, dtype, 3 if order == "mixed" else 0)
    w, bias, ad = layer(N + r, N, K, G, r, adtype)
    ids = numbers(M, M, G, order)
    q = cim.mxfp4_quantize_nhwc(w)
    b = bias if order == "mixed" else None
    y, tol, h, dh = want_forward(x, w, b, ad, ids, out)
    got = cim.mxfp4_linear_adapters_nhwc(x, q, b, ad, ids, out_dtype=out)
    ref.check(got, y, tol, "out")
    got, k, gh = cim.mxfp4_linear_adapters_nhwc(x, q, b, ad, ids, out_dtype=out, save=True)
    ref.check(got, y, tol, "out of the call that keeps")
    ref.check(gh, h, dh + 1e-40, "h")
    codes, scales, _, _ = kept.quantize(f64(x))
    assert np.array_equal(k.codes.cpu().numpy(), codes) and np.array_equal(k.scales.cpu().numpy(), scales)


BACKWARD = [(1, 1, 1, 1, 1), (1, 40, 33, 2, 5), (3, 70, 513, 5, 17), (33, 48, 64, 3, 16), (64, 130, 100, 4, 70), (129, 257, 130, 2, 40),
            (257, 60, 72, 4, 16), (300, 64, 64, 7, 20), (777, 100, 72, 3, 8), (1700, 264, 40, 3, 24), (2300, 40, 200, 3, 16),
            (5000, 33, 30, 2, 33)]


@pytest.mark.parametrize("M,N,K,G,r", BACKWARD)
@pytest.mark.parametrize("dtype,adtype,grad,out", [(BF16, BF16, BF16, BF16), (FP32, FP32, FP32, FP32), (FP16, FP16, FP16, FP32),
                                                   ("kept", BF16, BF16, BF16), ("kept", FP32, FP32, FP32)])
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_backward(M, N, K, G, r, dtype, adtype, grad, out, order):
    w, _, ad = layer(N + r, N, K, G, r, adtype)
    ids = numbers(M, M, G, order)
    dy = rows(M, M, N, grad, 5 if order == "mixed" else 0)
    x = rows(M + K, M, K, BF16 if dtype == "kept" else dtype, 3 if order == "mixed" else 0)
    if dtype == "kept":
        x = cim.mxint8_quantize_nhwc(x)
        x64 = kept.values(x)
    else:
        x64 = f64(x)
    g = np.random.default_rng(9)
    h = torch.from_numpy(g.standard_normal((M, r)).astype(np.float32)).cuda()
    wt = cim.mxfp4_quantize_nhwc(w, transpose=True)
    dx, ddown, dup = cim.mxfp4_linear_adapters_bwd_nhwc(dy, x, wt, ad, ids, h, dx_dtype=out)
    a, q, n = ref.mx_quantize(f64(dy))[2], ref.mx_quantize(f64(w).T)[2], f64(ids).astype(np.int64)
    mags = np.abs(a) @ np.abs(q).T
    down, up, scale = (f64(t) for t in ad)
    y, tol, t, dt = kept.beside(a @ q.T, (N / 32 + 40) * U * mags, mags, f64(dy), up, down, scale, n, out)
    ref.check(dx, y, tol, "dx")
    ref.check(ddown, *kept.grads(t, dt, x64, scale, n), "ddown")
    ref.check(dup, *kept.grads(f64(h), 0 * f64(h), f64(dy), scale, n), "dup")
    none, d2, u2 = cim.mxfp4_linear_adapters_bwd_nhwc(dy, x, None, ad, ids, h)
    assert none is None and torch.equal(d2, ddown) and torch.equal(u2, dup)


@pytest.mark.parametrize("G", [1, 3])
def test_no_row_has_an_adapter(G):
    for M in (1, 4, 40, 200, 300):
        x = rows(1, M, 96, BF16)
        w, bias, ad = layer(2, 64, 96, G, 16, BF16)
        q = cim.mxfp4_quantize_nhwc(w)
        ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
        got, _, h = cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad, ids, out_dtype=FP32, save=True)
        assert torch.equal(got, cim.mxfp4_linear_nhwc(x, q, bias, out_dtype=FP32)) and not h.any()
        assert torch.equal(got, cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad, ids, out_dtype=FP32))
        dy = rows(3, M, 64, BF16)
        wt = cim.mxfp4_quantize_nhwc(w, transpose=True)
        dx, ddown, dup = cim.mxfp4_linear_adapters_bwd_nhwc(dy, x, wt, ad, ids, h, dx_dtype=FP32)
        assert torch.equal(dx, cim.mxfp4_linear_nhwc(dy, wt, None, out_dtype=FP32)) and not ddown.any() and not dup.any()


@pytest.mark.parametrize("M", [200, 300])
@pytest.mark.parametrize("G,last", [(1, 111), (3, 111), (3, 101)])
def test_only_some_rows_have_an_adapter(M, G, last):
    """Whole tiles of rows without one, and an adapter with one row: the others are the layer's alone."""
    x, dy = rows(1, M, 96, BF16), rows(3, M, 64, BF16)
    w, bias, ad = layer(2, 64, 96, G, 16, BF16)
    q, wt = cim.mxfp4_quantize_nhwc(w), cim.mxfp4_quantize_nhwc(w, transpose=True)
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[100:last] = G - 1
    y, tol, h, dh = want_forward(x, w, bias, ad, ids, FP32)
    got, _, gh = cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad, ids, out_dtype=FP32, save=True)
    ref.check(got, y, tol, "out")
    ref.check(gh, h, dh + 1e-40, "h")
    none = ids < 0
    assert torch.equal(got[none], cim.mxfp4_linear_nhwc(x, q, bias, out_dtype=FP32)[none]) and not gh[none].any()
    dx, ddown, dup = cim.mxfp4_linear_adapters_bwd_nhwc(dy, x, wt, ad, ids, gh, dx_dtype=FP32)
    assert torch.equal(dx[none], cim.mxfp4_linear_nhwc(dy, wt, None, out_dtype=FP32)[none])
    n = f64(ids).astype(np.int64)
    t, dt = kept.through(f64(dy), f64(ad.up), n)
    ref.check(ddown, *kept.grads(t, dt, f64(x), f64(ad.scale), n), "ddown")
    ref.check(dup, *kept.grads(f64(gh), 0 * f64(gh), f64(dy), f64(ad.scale), n), "dup")


@pytest.mark.parametrize("M", [3, 40, 200, 300])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_infinities_stay_with_their_row_and_adapter(M, dtype):
    """Adapter 1 holds infinities and NaN and some rows do: only those rows, and rows of adapter 1, are not finite."""
    x = rows(1, M, 96, dtype)
    w, bias, ad = layer(2, 64, 96, 3, 16, dtype)
    q, wt = cim.mxfp4_quantize_nhwc(w), cim.mxfp4_quantize_nhwc(w, transpose=True)
    ids = torch.arange(M, dtype=torch.int32, device="cuda") % 4 - 1
    clean = cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad, ids, out_dtype=FP32, save=True)
    dy = rows(3, M, 64, dtype)
    grads = cim.mxfp4_linear_adapters_bwd_nhwc(dy, x, wt, ad, ids, clean[2], dx_dtype=FP32)
    bad = cim.Adapters(ad.down.clone(), ad.up.clone(), ad.scale)
    bad.down[1, 3, 5] = float("inf")
    bad.up[1, 2, 9] = float("nan")
    got = cim.mxfp4_linear_adapters_nhwc(x, q, bias, bad, ids, out_dtype=FP32, save=True)
    mine = ids == 1
    assert torch.equal(got[0][~mine], clean[0][~mine]) and torch.equal(got[2][~mine], clean[2][~mine])
    assert not torch.isfinite(got[0][mine]).any(1).all() and not torch.isfinite(got[2][mine]).all()
    assert torch.equal(cim.mxfp4_linear_adapters_nhwc(x, q, bias, bad, ids, out_dtype=FP32)[~mine], clean[0][~mine]) or M <= 64
    back = cim.mxfp4_linear_adapters_bwd_nhwc(dy, x, wt, bad, ids, clean[2], dx_dtype=FP32)
    assert torch.equal(back[0][~mine], grads[0][~mine])
    for k in (1, 2):
        assert torch.equal(back[k][0], grads[k][0]) and torch.equal(back[k][2], grads[k][2])
    x2, dy2 = x.clone(), dy.clone()
    x2[0, 7], dy2[0, 7] = float("nan"), float("inf")      # row 0 has no adapter
    got = cim.mxfp4_linear_adapters_nhwc(x2, q, bias, ad, ids, out_dtype=FP32, save=True)
    assert torch.equal(got[0][1:], clean[0][1:]) and torch.equal(got[2], clean[2])
    back = cim.mxfp4_linear_adapters_bwd_nhwc(dy2, x2, wt, ad, ids, clean[2], dx_dtype=FP32)
    assert torch.equal(back[0][1:], grads[0][1:]) and torch.equal(back[1], grads[1]) and torch.equal(back[2], grads[2])


@pytest.mark.parametrize("M", [200, 300])
def test_same_row_alone_and_in_a_batch(M):
    """A row's output is one adapter's, whatever else is in the batch."""
    w, bias, ad = layer(2, 96, 160, 6, 16, BF16)
    q = cim.mxfp4_quantize_nhwc(w)
    x = rows(1, M, 160, BF16)
    ids = numbers(1, M, 6, "mixed")
    every = cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad, ids, out_dtype=FP32)
    y, tol, _, _ = want_forward(x, w, bias, ad, ids, FP32)
    for k in (0, 3, 63, 64, 150, M - 1):
        one = cim.mxfp4_linear_adapters_nhwc(x[k:k + 1], q, bias, ad, ids[k:k + 1], out_dtype=FP32)
        assert (np.abs(f64(one) - f64(every[k:k + 1])) <= 2 * tol[k:k + 1]).all()


def test_maps_and_no_rows():
    w, bias, ad = layer(2, 40, 64, 3, 8, BF16)
    q, wt = cim.mxfp4_quantize_nhwc(w), cim.mxfp4_quantize_nhwc(w, transpose=True)
    x = rows(1, 70, 64, BF16).view(2, 7, 5, 64)
    ids = numbers(3, 70, 3, "mixed").view(2, 7, 5)
    out, k, h = cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad, ids, save=True)
    assert out.shape == (2, 7, 5, 40) and h.shape == (2, 7, 5, 8) and k.rows == 70
    flat = cim.mxfp4_linear_adapters_nhwc(x.view(70, 64), q, bias, ad, ids.view(70), save=True)
    assert torch.equal(out.view(70, 40), flat[0]) and torch.equal(h.view(70, 8), flat[2])
    dy = rows(5, 70, 40, BF16).view(2, 7, 5, 40)
    dx, ddown, dup = cim.mxfp4_linear_adapters_bwd_nhwc(dy, k, wt, ad, ids, h)
    assert dx.shape == x.shape
    out, k, h = cim.mxfp4_linear_adapters_nhwc(x[:0], q, bias, ad, ids[:0], save=True)
    assert out.shape == (0, 7, 5, 40) and h.shape == (0, 7, 5, 8)
    dx, ddown, dup = cim.mxfp4_linear_adapters_bwd_nhwc(dy[:0], k, wt, ad, ids[:0], h)
    assert dx.shape == (0, 7, 5, 64) and ddown.shape == ad.down.shape and not ddown.any() and not dup.any()
