"""MXFP4 rows and the linear layer on them on the GPU, against the
definitions in 64 bits (row_reference.py has them and the tolerances)."""
import numpy as np
import pytest
import torch

import convolution_implicit_gemm_fwd_amd as cim
import row_reference as ref
from gpu_harness import need_gpu
from row_reference import f64

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def rows(seed, n, cols, dtype, pad=0, offset=0, scale=1.0):
    """Normal values whose size changes from block to block, a row's start anywhere."""
    g = np.random.default_rng(seed)
    a = g.standard_normal((n, cols + pad)) * scale * np.exp2(g.integers(-3, 4, (n, cols + pad)) // 2)
    t = torch.from_numpy(a.astype(np.float32)).to(dtype)
    flat = torch.empty(t.numel() + offset, dtype=dtype, device="cuda")
    flat[offset:].copy_(t.reshape(-1))
    return flat[offset:].view(n, cols + pad)[:, :cols]


def same_packed(q, x64):
    codes, scales, _, bad = ref.mx_quantize(x64)
    got = q.codes.cpu().numpy().reshape(codes.shape[0], -1, 16)
    want = codes.reshape(got.shape)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(got[~bad], want[~bad])      # the codes of a block without a scale mean nothing


SIZES = [(1, 1), (1, 32), (3, 33), (40, 64), (7, 100), (33, 129), (5, 511), (130, 640), (64, 1000), (2, 4096), (1, 9000),
         (513, 96), (300, 300)]


@pytest.mark.parametrize("n,cols", SIZES)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantize(n, cols, dtype, pad, offset, transpose):
    x = rows(n + cols, n, cols, dtype, pad, offset)
    q = cim.mxfp4_quantize_nhwc(x, transpose=transpose)
    a = f64(x)
    same_packed(q, a.T if transpose else a)


@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_every_rounding(transpose):
    """Every grid value, every tie and the values just beside, with blocks of each size and sign; zeros; the largest and
    smallest numbers of each type."""
    g = ref.GRID
    marks = np.concatenate([g, (g[1:] + g[:-1]) / 2, [5, 7, 7.984375]])
    marks = np.unique(np.concatenate([marks, marks * (1 - 2.0 ** -7), marks * (1 + 2.0 ** -7), [0.0]]))
    marks = marks[marks < 8]
    line = np.concatenate([marks, -marks])
    blocks = []
    for e in (-120, -40, -1, 0, 9, 100):
        for k in range(0, len(line), 31):
            b = np.zeros(32)
            b[:len(line[k:k + 31])] = line[k:k + 31]
            b[31] = 4.0
            blocks.append(b * 2.0 ** e)
    blocks.append(np.zeros(32))
    blocks.append(-np.zeros(32))
    top = np.full(32, 2.0 ** 127 * 1.9921875)
    blocks += [top, np.concatenate([[2.0 ** -126, -2.0 ** -127, 2.0 ** -128], np.zeros(29)]),
               np.concatenate([[2.0 ** -133], np.zeros(31)])]
    a = np.stack(blocks).astype(np.float32)
    for t in (torch.from_numpy(a), torch.from_numpy(a).to(BF16), torch.from_numpy(np.clip(a, -65504, 65504)).to(FP16)):
        x = t.cuda()
        q = cim.mxfp4_quantize_nhwc(x.t().contiguous() if transpose else x, transpose=transpose)
        same_packed(q, f64(x))


@pytest.mark.parametrize("transpose", [False, True])
def test_blocks_with_nan_or_infinity_stand_for_nan(transpose):
    x = rows(3, 40, 100, FP32)
    x[1, 5], x[2, 40], x[3, 99], x[39, 0] = float("nan"), float("inf"), float("-inf"), float("nan")
    v = x.t().contiguous() if transpose else x
    q = cim.mxfp4_quantize_nhwc(v, transpose=transpose)
    same_packed(q, f64(x))
    d = f64(cim.mxfp4_dequantize_nhwc(q, FP32))
    want = ref.mx_quantize(f64(x))[2]
    assert np.array_equal(d, want, equal_nan=True)
    w = cim.mxfp4_quantize_nhwc(rows(4, 50, 100, FP32))
    y = f64(cim.mxfp4_linear_nhwc(q, w, out_dtype=FP32))
    hit = [1, 2, 3, 39]
    assert np.isnan(y[hit]).all() and np.isfinite(np.delete(y, hit, 0)).all()
    y = f64(cim.mxfp4_linear_nhwc(x[:3], w, out_dtype=FP32))      # a few rows
    assert np.isnan(y[1:]).all() and np.isfinite(y[0]).all()


@pytest.mark.parametrize("n,cols", SIZES)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_dequantize(n, cols, dtype):
    x = rows(cols, n, cols, FP32)
    q = cim.mxfp4_quantize_nhwc(x)
    want = ref.mx_quantize(f64(x))[2]
    ref.check(cim.mxfp4_dequantize_nhwc(q, dtype), want, 0, "values")      # the grid and these scales fit every type


def test_empty():
    x = torch.empty(0, 64, device="cuda")
    q = cim.mxfp4_quantize_nhwc(x)
    assert q.codes.numel() == 0 and cim.mxfp4_dequantize_nhwc(q, FP32).shape == (0, 64)
    w = cim.mxfp4_quantize_nhwc(rows(1, 8, 64, FP32))
    assert cim.mxfp4_linear_nhwc(x, w).shape == (0, 8) and cim.mxfp4_linear_nhwc(q, w).shape == (0, 8)
    dx, dw, db = cim.mxfp4_linear_bwd_nhwc(torch.empty(0, 8, device="cuda"), x, rows(1, 8, 64, FP32))
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def check_linear(M, N, K, xt, out, bias=True, pad=0, offset=0, packed=False):
    x, w = rows(M + K, M, K, xt, pad, offset), rows(N, N, K, FP32, scale=K ** -0.5)
    b = torch.from_numpy(np.random.default_rng(N).standard_normal(N).astype(np.float32)).cuda() if bias else None
    q = cim.mxfp4_quantize_nhwc(w)
    got = cim.mxfp4_linear_nhwc(cim.mxfp4_quantize_nhwc(x) if packed else x, q, b, out_dtype=out)
    y, tol = ref.product(ref.mx_quantize(f64(x))[2], ref.mx_quantize(f64(w))[2], f64(b) if bias else None, out)
    ref.check(got, y, tol, "linear %d %d %d" % (M, N, K))


@pytest.mark.parametrize("M", [1, 2, 5, 15, 16, 17, 31, 33, 48, 64, 65, 100, 128, 129, 200, 257])
@pytest.mark.parametrize("N,K", [(1, 1), (16, 32), (50, 100), (64, 512), (129, 130), (272, 1056), (40, 2500), (1000, 300)])
def test_linear(M, N, K):
    check_linear(M, N, K, BF16, BF16)
    check_linear(M, N, K, FP32, FP32, bias=False, packed=True)


@pytest.mark.parametrize("M,N,K", [(1, 100, 260), (20, 100, 260), (90, 100, 260), (300, 300, 260)])
@pytest.mark.parametrize("xt", [BF16, FP16, FP32])
@pytest.mark.parametrize("out", [BF16, FP16, FP32])
def test_linear_types_and_strides(M, N, K, xt, out):
    check_linear(M, N, K, xt, out)
    check_linear(M, N, K, xt, out, pad=5, offset=1)
    check_linear(M, N, K, xt, out, packed=True)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (7, 2048, 8192), (520, 768, 640), (1024, 1024, 2048), (700, 2050, 1000),
                                   (2100, 260, 160), (3136, 512, 512), (4096, 2304, 256)])
def test_linear_large(M, N, K):
    check_linear(M, N, K, BF16, FP32)


def test_linear_on_a_map():
    x = rows(1, 2 * 3 * 5, 64, BF16).view(2, 3, 5, 64)
    w = cim.mxfp4_quantize_nhwc(rows(2, 48, 64, FP32))
    y = cim.mxfp4_linear_nhwc(x, w)
    assert y.shape == (2, 3, 5, 48) and y.dtype == BF16
    assert torch.equal(y.view(-1, 48), cim.mxfp4_linear_nhwc(x.view(-1, 64), w))


def check_bwd(M, N, K, grad, t, out, pad=0, offset=0):
    dy, x, w = rows(1, M, N, grad, pad, offset, 0.1), rows(2, M, K, t, pad, offset), rows(3, N, K, t, pad, offset, 0.1)
    dx, dw, db = cim.mxfp4_linear_bwd_nhwc(dy, x, w, dx_dtype=out)
    q = lambda a: ref.mx_quantize(a)[2]      # noqa: E731
    a, tol = ref.product(q(f64(dy)), q(f64(w).T), None, out)
    ref.check(dx, a, tol, "dx")
    a, tol = ref.product(q(f64(dy).T), q(f64(x).T), None, FP32)
    ref.check(dw, a, tol, "dw")
    g = f64(dy)
    ref.check(db, g.sum(0), (-(-M // 128) + 128 + 16) * ref.U * np.abs(g).sum(0), "db")


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 40, 70), (31, 32, 33), (64, 64, 64), (100, 130, 50), (257, 96, 300),
                                   (1000, 70, 130), (2500, 520, 260)])
@pytest.mark.parametrize("grad,t,out", [(BF16, BF16, BF16), (FP32, FP16, FP32), (FP16, FP32, BF16)])
def test_backward(M, N, K, grad, t, out):
    check_bwd(M, N, K, grad, t, out)
    check_bwd(M, N, K, grad, t, out, pad=3, offset=1)


def test_backward_against_differences():
    """On values that 4 bits hold exactly the layer is linear in x and in w, so central differences of the forward
    definition are its gradient."""
    g = np.random.default_rng(5)
    M, N, K = 64, 32, 96

    def grid(n, k):
        a = g.choice(np.concatenate([ref.GRID, -ref.GRID]), (n, k))
        a[::32, :], a[:, ::32] = 6, 6            # every block, either way, has the same scale
        return a

    dy, x, w = grid(M, N), grid(M, K), grid(N, K)
    to = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()      # noqa: E731
    dx, dw, db = (f64(t) for t in cim.mxfp4_linear_bwd_nhwc(to(dy), to(x), to(w)))
    loss = lambda x, w, b: ((x @ w.T + b) * dy).sum()      # noqa: E731
    zero = np.zeros(N)
    for k in range(0, M * K, 97):
        e = np.zeros((M, K))
        e.reshape(-1)[k] = 0.5
        assert dx.reshape(-1)[k] == loss(x + e, w, zero) - loss(x - e, w, zero)
    for k in range(0, N * K, 61):
        e = np.zeros((N, K))
        e.reshape(-1)[k] = 0.5
        assert dw.reshape(-1)[k] == loss(x, w + e, zero) - loss(x, w - e, zero)
    for k in range(N):
        e = np.zeros(N)
        e[k] = 0.5
        assert db[k] == loss(x, w, e) - loss(x, w, -e)


def test_repeats_bit_for_bit():
    for M in (3, 40, 600):
        x, w = rows(1, M, 1100, BF16), cim.mxfp4_quantize_nhwc(rows(2, 300, 1100, FP32))
        first = cim.mxfp4_linear_nhwc(x, w, out_dtype=FP32)
        for _ in range(3):
            assert torch.equal(first, cim.mxfp4_linear_nhwc(x, w, out_dtype=FP32))


def test_refusals():
    x = rows(1, 8, 64, BF16)
    w = cim.mxfp4_quantize_nhwc(rows(2, 16, 96, FP32))
    with pytest.raises(ValueError):
        cim.mxfp4_linear_nhwc(x, w)                              # 64 columns for 96
    with pytest.raises(TypeError):
        cim.mxfp4_quantize_nhwc(x.to(torch.float64))
    with pytest.raises(ValueError):
        cim.mxfp4_linear_nhwc(rows(1, 8, 96, BF16), w, torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        cim.mxfp4_quantize_nhwc(x.t())                           # columns apart
    with pytest.raises(ValueError):
        cim.mxfp4_dequantize_nhwc(w._replace(cols=64), BF16)
    with pytest.raises(ValueError):
        cim.layer_norm_nhwc(x, torch.ones(64, device="cuda", dtype=BF16))
    with pytest.raises(ValueError):
        cim.layer_norm_bwd_nhwc(x[:4], x, None, x[:, 0].float(), x[:, 0].float())
    with pytest.raises(TypeError):
        cim.mxfp4_linear_bwd_nhwc(rows(3, 8, 16, BF16), x, rows(2, 16, 64, FP32))


def side_stream_cases():
    x, w, dy = rows(1, 300, 256, BF16), rows(2, 128, 256, BF16), rows(3, 300, 128, BF16)
    q = cim.mxfp4_quantize_nhwc(w)
    mean, rstd = cim.layer_norm_nhwc(x, stats=True)[1:]
    return [lambda **s: cim.layer_norm_nhwc(x, stats=True, **s), lambda **s: tuple(cim.layer_norm_mxfp4_nhwc(x, **s))[:2],
            lambda **s: cim.layer_norm_bwd_nhwc(x, x, None, mean, rstd, **s),
            lambda **s: tuple(cim.mxfp4_quantize_nhwc(x, transpose=True, **s))[:2],
            lambda **s: (cim.mxfp4_dequantize_nhwc(q, FP32, **s),), lambda **s: (cim.mxfp4_linear_nhwc(x, q, **s),),
            lambda **s: (cim.mxfp4_linear_nhwc(x[:9], q, **s),), lambda **s: cim.mxfp4_linear_bwd_nhwc(dy, x, w, **s)]


def test_another_stream():
    """On a stream that is held back, a call's buffers are not handed out again before it has run."""
    for call in side_stream_cases():
        want = call()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = call(stream=side.cuda_stream)
        junk = [torch.full((1 << k,), 0xFF, dtype=torch.uint8, device="cuda") for k in range(9, 21) for _ in range(2)]
        torch.cuda.synchronize()
        del junk
        for p, q in zip(got, want):
            assert torch.equal(p, q)


def test_graph_replays():
    """Captured once, replayed between eager work: every replay equals the eager result on the inputs it finds."""
    x, w, dy = rows(1, 200, 160, BF16), rows(2, 96, 160, BF16), rows(3, 200, 96, BF16)
    q = cim.mxfp4_quantize_nhwc(w)

    def step():
        y, mean, rstd = cim.layer_norm_nhwc(x, stats=True)
        z = cim.mxfp4_linear_nhwc(y, q)
        one = cim.mxfp4_linear_nhwc(y[:1], q)
        g = cim.mxfp4_linear_bwd_nhwc(dy, y, w)
        n = cim.layer_norm_bwd_nhwc(g[0], x, None, mean, rstd)
        return (y, mean, rstd, z, one, *g, *n)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(rows(10 + k, 200, 160, BF16))
        dy.copy_(rows(20 + k, 200, 96, BF16))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for p, e in zip(got, step()):
            assert torch.equal(p, e), "replay %d" % k
