"""The passes on activations kept in 8 bits and the low-rank adapters as a program calls them, on the GPU: streams,
captured graphs, repeats, the compiled calls, refusals, the edges of their variants and of 32-bit offsets."""
import numpy as np
import pytest
import torch

import convolution_implicit_gemm_fwd_amd as cim
import kept_reference as kept
import row_reference as ref
from convolution_implicit_gemm_fwd_amd import rows as R
from gpu_harness import need_gpu
from row_reference import U, f64
from test_gpu_adapters import layer, numbers, want_forward
from test_gpu_mxfp4 import rows

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def flat(r):
    return [r] if isinstance(r, torch.Tensor) else [t for v in r if v is not None and not isinstance(v, int) for t in flat(v)]


def calls():
    """Each entry point, in each of its ways through the kernels."""
    out = []
    x, dy = rows(1, 300, 256, BF16), rows(3, 300, 128, BF16)
    gamma = torch.rand(256, device="cuda") + 0.5
    q8 = cim.mxint8_quantize_nhwc(x)
    y, k8, rstd = cim.layer_norm_mxint8_nhwc(x, gamma)
    w, bias, ad = layer(2, 128, 256, 5, 20, BF16)
    q, wt = cim.mxfp4_quantize_nhwc(w), cim.mxfp4_quantize_nhwc(w, transpose=True)
    ids, wb = numbers(4, 300, 5, "mixed"), w.bfloat16()      # (held: the caller keeps a call's inputs until it has run)
    out += [lambda **s: cim.mxint8_quantize_nhwc(x, **s), lambda **s: cim.mxint8_dequantize_nhwc(q8, FP16, **s),
            lambda **s: cim.layer_norm_mxint8_nhwc(x, gamma, **s), lambda **s: cim.layer_norm_bwd_mxint8_nhwc(x, k8, gamma, rstd, **s),
            lambda **s: cim.mxfp4_linear_bwd_nhwc(dy, q8, wb, **s)]
    for m in (1, 4, 30, 300):
        for save in (False, True):
            out.append(lambda m=m, save=save, **s: cim.mxfp4_linear_adapters_nhwc(x[:m], q, bias, ad, ids[:m], save=save, **s))
        h = cim.mxfp4_linear_adapters_nhwc(x[:m], q, bias, ad, ids[:m], save=True)[2]
        k = cim.mxint8_quantize_nhwc(x[:m])
        out += [lambda m=m, h=h, k=k, **s: cim.mxfp4_linear_adapters_bwd_nhwc(dy[:m], k, wt, ad, ids[:m], h, **s),
                lambda m=m, h=h, **s: cim.mxfp4_linear_adapters_bwd_nhwc(dy[:m], x[:m], wt, ad, ids[:m], h, FP32, **s)]
    return out


def test_repeats_bit_for_bit():
    for k, call in enumerate(calls()):
        first = flat(call())
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, flat(call()))), "call %d" % k


def test_another_stream():
    """On a stream that is held back, a call's buffers are not handed out again before it has run."""
    for k, call in enumerate(calls()):
        want = [t.clone() for t in flat(call())]
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(10_000_000)
        got = flat(call(stream=side.cuda_stream))
        junk = [torch.full((1 << b,), 0xFF, dtype=torch.uint8, device="cuda") for b in range(9, 21) for _ in range(2)]
        torch.cuda.synchronize()
        del junk
        assert all(torch.equal(a, b) for a, b in zip(got, want)), "call %d" % k


def test_two_calls_at_once():
    w, bias, ad = layer(2, 512, 512, 5, 24, BF16)
    q, wt = cim.mxfp4_quantize_nhwc(w), cim.mxfp4_quantize_nhwc(w, transpose=True)
    jobs = []
    for k in range(4):
        x, dy, ids = rows(k, 900, 512, BF16), rows(k + 9, 900, 512, BF16), numbers(k, 900, 5, "mixed")

        def job(x=x, dy=dy, ids=ids, **s):
            _, k8, h = cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad, ids, save=True, **s)
            return cim.mxfp4_linear_adapters_bwd_nhwc(dy, k8, wt, ad, ids, h, **s)
        jobs.append((job, job()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(3):
        got = [job(stream=s.cuda_stream) for (job, _), s in zip(jobs, streams)]
        torch.cuda.synchronize()
        for (_, want), r in zip(jobs, got):
            assert all(torch.equal(a, b) for a, b in zip(want, r))


def test_graph_replays():
    """A training step captured once and replayed between eager work: every replay equals the eager result on the inputs
    that it finds, other adapters a row among them; two graphs do not share what they write."""
    w, bias, ad = layer(2, 96, 160, 5, 16, BF16)
    q, wt = cim.mxfp4_quantize_nhwc(w), cim.mxfp4_quantize_nhwc(w, transpose=True)
    gamma = torch.rand(160, device="cuda") + 0.5
    x, dy, ids = rows(1, 300, 160, BF16), rows(3, 300, 96, BF16), numbers(1, 300, 5, "mixed")

    def step(m):
        y, n8, rstd = cim.layer_norm_mxint8_nhwc(x[:m], gamma)
        z, y8, h = cim.mxfp4_linear_adapters_nhwc(y, q, bias, ad, ids[:m], save=True)
        g = cim.mxfp4_linear_adapters_bwd_nhwc(dy[:m], y8, wt, ad, ids[:m], h)
        full = cim.mxfp4_linear_bwd_nhwc(dy[:m], y8, w.bfloat16())
        return flat((y, n8, rstd, z, y8, h, g, full, cim.layer_norm_bwd_mxint8_nhwc(g[0], n8, gamma, rstd),
                     cim.mxint8_dequantize_nhwc(y8, BF16), cim.mxfp4_linear_adapters_nhwc(y[:2], q, None, ad, ids[:2])))

    graphs = []
    for m in (300, 200, 40):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(m)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(m)
        graphs.append((m, graph, out))
    for k in range(4):
        x.copy_(rows(10 + k, 300, 160, BF16))
        dy.copy_(rows(20 + k, 300, 96, BF16))
        ids.copy_(numbers(30 + k, 300, 5, "mixed" if k % 2 else "runs"))
        for _, graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for m, _, out in graphs:
            got = [t.clone() for t in out]
            for i, (p, e) in enumerate(zip(got, step(m))):
                assert torch.equal(p, e), "replay %d of %d rows, tensor %d" % (k, m, i)


class Left:
    """Leaves every call to Python."""

    def __getattr__(self, name):
        return lambda *a: None


def test_same_results_as_in_python(monkeypatch):
    for k, call in enumerate(calls()):
        taken = []

        class Seen:
            def __getattr__(self, name, fast=R._fast):
                f = getattr(fast, name)
                return lambda *a: taken.append(f(*a)) or taken[-1]

        with monkeypatch.context() as m:
            m.setattr(R, "_fast", Seen())
            one = call()
        assert taken and all(r is not None for r in taken), "call %d is not taken" % k
        with monkeypatch.context() as m:
            m.setattr(R, "_fast", Left())
            two = call()
        assert type(one) is type(two) and [type(v) for v in one] == [type(v) for v in two]
        for a, b in zip(flat(one), flat(two)):
            assert a.shape == b.shape and a.dtype == b.dtype and a.is_contiguous() and torch.equal(a, b), "call %d" % k


def test_uncommon_tensors():
    """Rows apart in three dimensions, one vector, strided statistics."""
    w, bias, ad = layer(2, 40, 64, 3, 8, FP32)
    q = cim.mxfp4_quantize_nhwc(w)
    x = torch.randn(4, 6, 80, device="cuda")[:, :1, :64]
    ids = torch.tensor([[2], [-1], [0], [2]], dtype=torch.int32, device="cuda")
    got = cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad, ids, save=True)
    want = cim.mxfp4_linear_adapters_nhwc(x.contiguous(), q, bias, ad, ids, save=True)
    assert all(torch.equal(a, b) for a, b in zip(flat(got), flat(want))) and got[0].shape == (4, 1, 40)
    one = cim.mxfp4_linear_adapters_nhwc(x[3, 0], q, bias, ad, ids[3, 0], save=True)
    assert one[0].shape == (40,) and one[2].shape == (8,)
    y, k8, rstd = cim.layer_norm_mxint8_nhwc(x)
    twice = torch.stack((rstd, rstd), -1)[..., 0]
    assert not twice.is_contiguous()
    assert all(torch.equal(a, b) for a, b in zip(cim.layer_norm_bwd_mxint8_nhwc(x, k8, None, twice),
                                                 cim.layer_norm_bwd_mxint8_nhwc(x.contiguous(), k8, None, rstd)))
    p = torch.nn.Parameter(ad.down)
    assert torch.equal(cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad._replace(down=p), ids), got[0])


def test_refusals():
    x = rows(1, 8, 64, BF16)
    w, bias, ad = layer(2, 40, 64, 3, 8, BF16)
    q, ids = cim.mxfp4_quantize_nhwc(w), torch.zeros(8, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad, ids.cpu())
    with pytest.raises(ValueError):
        cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad, ids.long())
    with pytest.raises(ValueError):
        cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad._replace(scale=ad.scale.cpu()), ids)
    with pytest.raises(ValueError):
        cim.mxfp4_linear_adapters_nhwc(cim.mxfp4_quantize_nhwc(x)[0].view(8, 32), q, bias, ad, ids)
    with pytest.raises(RuntimeError, match="status 4"):
        big = cim.Adapters(torch.zeros(1, 4097, 64, device="cuda"), torch.zeros(1, 4097, 40, device="cuda"), torch.ones(1, device="cuda"))
        cim.mxfp4_linear_adapters_nhwc(x, q, bias, big, ids)
    k8 = cim.mxint8_quantize_nhwc(x)
    with pytest.raises(RuntimeError, match="status 13"):      # codes that do not start at 16 bytes
        cim.mxint8_dequantize_nhwc(k8._replace(codes=torch.zeros(8 * 64 + 1, dtype=torch.int8, device="cuda")[1:].view(8, 64)), FP32)


@pytest.mark.parametrize("M,N,K", [(3, 64, 2048), (40, 64, 2048), (61, 6200, 1100), (256, 6200, 1100), (600, 520, 300),
                                   (2500, 2600, 200), (3100, 3100, 600)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_infinities_in_every_product(M, N, K, dtype):
    """One per shape of the product, those whose wave groups share a tile's adapters among them: an infinity and a NaN in
    up reach their own columns of their own adapter's rows, exactly, and change nothing else."""
    x = rows(1, M, K, dtype)
    w, bias, ad = layer(2, N, K, 5, 40, dtype)
    q = cim.mxfp4_quantize_nhwc(w)
    ids = numbers(7, M, 5, "mixed")
    ids[0] = 1
    clean = cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad, ids, out_dtype=FP32, save=True)
    up = ad.up.clone()
    up[1, 33, 9], up[1, 2, 31], up[1, 2, N - 1] = float("inf"), float("nan"), float("-inf")
    got = cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad._replace(up=up), ids, out_dtype=FP32)
    mine = ids == 1
    assert torch.equal(got[~mine], clean[0][~mine])
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[[9, 31, N - 1]] = False
    assert torch.equal(got[mine][:, rest], clean[0][mine][:, rest])
    h = clean[2][mine]
    assert torch.equal(got[mine, 9], torch.where(h[:, 33] > 0, 1.0, -1.0) * float("inf"))
    assert torch.equal(got[mine, N - 1], torch.where(h[:, 2] > 0, -1.0, 1.0) * float("inf"))
    assert got[mine, 31].isnan().all()


@pytest.mark.parametrize("M,N,K,G,r", [(1030, 96, 1030, 3, 16), (1100, 130, 640, 300, 16), (2000, 64, 200, 700, 5),
                                       (4100, 520, 260, 2, 64), (8200, 64, 130, 40, 24), (1500, 72, 2600, 3, 100)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_forward_at_the_edges_of_its_variants(M, N, K, G, r, dtype):
    """Rows sorted by one and by two digits, many and few adapters a tile, every number of ranks a workgroup."""
    x = rows(M, M, K, dtype, 3)
    w, bias, ad = layer(N, N, K, G, r, dtype)
    ids = numbers(M, M, G, "mixed")
    y, tol, h, dh = want_forward(x, w, bias, ad, ids, FP32)
    got, _, gh = cim.mxfp4_linear_adapters_nhwc(x, cim.mxfp4_quantize_nhwc(w), bias, ad, ids, out_dtype=FP32, save=True)
    ref.check(got, y, tol, "out")
    ref.check(gh, h, dh + 1e-40, "h")


@pytest.mark.parametrize("M,N,K,G,r", [(1100, 130, 64, 300, 16), (2000, 64, 200, 700, 5), (9000, 40, 130, 2, 24),
                                       (300, 72, 260, 1, 100), (20000, 33, 40, 3, 8)])
def test_gradients_at_the_edges_of_their_variants(M, N, K, G, r):
    """One row an adapter, adapters over many chunks of rows, an adapter with nearly all rows."""
    w, _, ad = layer(N, N, K, G, r, BF16)
    ids = numbers(M, M, G, "mixed")
    if G == 2:
        ids = torch.where(torch.arange(M, device="cuda") % 50 == 7, 0, 1).int()
    dy, x = rows(1, M, N, BF16), rows(2, M, K, FP32)
    h = torch.from_numpy(np.random.default_rng(9).standard_normal((M, r)).astype(np.float32)).cuda()
    _, ddown, dup = cim.mxfp4_linear_adapters_bwd_nhwc(dy, x, None, ad, ids, h)
    n = f64(ids).astype(np.int64)
    t, dt = kept.through(f64(dy), f64(ad.up), n)
    ref.check(ddown, *kept.grads(t, dt, f64(x), f64(ad.scale), n), "ddown")
    ref.check(dup, *kept.grads(f64(h), 0 * f64(h), f64(dy), f64(ad.scale), n), "dup")


def test_gradients_by_differences():
    """The adapters' part is linear in x, in down and in up: central differences of its definition are its gradients."""
    g = np.random.default_rng(5)
    M, N, K, G, r = 37, 64, 96, 3, 8
    whole = lambda *s: g.integers(-4, 5, s).astype(np.float64)      # noqa: E731 (products and sums are exact)
    x, down, up, dy = whole(M, K), whole(G, r, K), whole(G, r, N), whole(M, N)
    scale, ids = np.array([0.5, 1.0, 2.0]), g.integers(-1, 3, M)
    to = lambda a, t=FP32: torch.from_numpy(a).to(t).cuda()      # noqa: E731

    def loss(x, down, up):
        return sum(scale[i] * ((x[m] @ down[i].T @ up[i]) * dy[m]).sum() for i in range(G) for m in [ids == i])
    h = np.zeros((M, r))
    for i in range(G):
        h[ids == i] = x[ids == i] @ down[i].T
    zero = cim.mxfp4_quantize_nhwc(torch.zeros(K, N, device="cuda"))
    ad = cim.Adapters(to(down, BF16), to(up, BF16), to(scale))
    dx, ddown, dup = (f64(t) for t in cim.mxfp4_linear_adapters_bwd_nhwc(to(dy), to(x), zero, ad, to(ids, torch.int32), to(h)))
    for grad, k in ((dx, 0), (ddown, 1), (dup, 2)):
        for at in range(0, grad.size, 53):
            a = [x, down, up]
            e = np.zeros(a[k].shape)
            e.reshape(-1)[at] = 1
            plus, minus = list(a), list(a)
            plus[k], minus[k] = a[k] + e, a[k] - e
            assert grad.reshape(-1)[at] == (loss(*plus) - loss(*minus)) / 2


def test_past_32_bit_offsets():
    """Kept rows of more than 2^32 bytes, rows of x 2^31 elements and more apart from the first, adapters past 2^32 bytes."""
    n, cols = (1 << 20) + 3, 4160
    x = torch.zeros(n, cols, dtype=BF16, device="cuda")
    x[-5:] = rows(1, 5, cols, BF16)
    q = cim.mxint8_quantize_nhwc(x)
    codes, scales, val, _ = kept.quantize(f64(x[-5:]))
    assert q.codes.numel() > 1 << 32
    assert np.array_equal(q.codes[-5:].cpu().numpy(), codes) and np.array_equal(q.scales[-5:].cpu().numpy(), scales)
    del x
    back = cim.mxint8_dequantize_nhwc(q, BF16)
    assert np.array_equal(f64(back[-5:]), val)
    y, k8, rstd = cim.layer_norm_mxint8_nhwc(back)
    nn, _, dn, _ = kept.norm(val, 1e-5)
    kept.check_kept(cim.Mxint8Tensor(k8.codes[-5:], k8.scales[-5:], 5, cols), nn, dn, "kept")
    dx, _, _ = cim.layer_norm_bwd_mxint8_nhwc(back, k8, None, rstd)
    w = kept.norm_bwd(val, kept.values(cim.Mxint8Tensor(k8.codes[-5:], k8.scales[-5:], 5, cols)), None, f64(rstd[-5:]), BF16)
    ref.check(dx[-5:], w[0], w[3], "dx")


def test_adapters_past_32_bit_offsets():
    G, r, K, N = 70000, 16, 2048, 40      # down 4.6 GB
    down = torch.zeros(G, r, K, dtype=BF16, device="cuda")
    w, bias, some = layer(3, N, K, 2, r, BF16)
    down[-1], down[-2] = some.down[0], some.down[1]
    up = torch.zeros(G, r, N, dtype=BF16, device="cuda")
    up[-1], up[-2] = some.up[0], some.up[1]
    ad = cim.Adapters(down, up, torch.full((G,), 1.5, device="cuda"))
    small = cim.Adapters(some.down, some.up, torch.full((2,), 1.5, device="cuda"))
    q = cim.mxfp4_quantize_nhwc(w)
    for M in (2, 40, 1500):
        x = rows(M, M, K, BF16)
        two = torch.arange(M, dtype=torch.int32, device="cuda") % 3 - 1      # -1, 0, 1
        ids = torch.where(two < 0, -1, G - 1 - two).int()
        got = cim.mxfp4_linear_adapters_nhwc(x, q, bias, ad, ids, out_dtype=FP32, save=True)
        y, tol, h, dh = want_forward(x, w, bias, small, two, FP32)
        ref.check(got[0], y, tol, "out")
        ref.check(got[2], h, dh + 1e-40, "h")
        dy = rows(5, M, N, BF16)
        _, ddown, dup = cim.mxfp4_linear_adapters_bwd_nhwc(dy, x, None, ad, ids, got[2])
        t, dt = kept.through(f64(dy), f64(small.up), f64(two).astype(np.int64))
        want, tol = kept.grads(t, dt, f64(x), f64(small.scale), f64(two).astype(np.int64))
        ref.check(ddown[[G - 1, G - 2]], want, tol, "ddown")
        assert not ddown[:G - 2].any() and not dup[:G - 2].any()
        del ddown, dup


@pytest.mark.parametrize("dtype,low", [(BF16, -130), (FP16, -22), (FP32, -100)])
@pytest.mark.parametrize("M", [3, 40, 300])
def test_the_smallest_values(dtype, low, M):
    """Rows near and below the smallest normal value lose nothing: large adapters bring them back to ordinary sizes."""
    N, K, G, r = 64, 160, 3, 20
    up = 10 if dtype == FP16 else 100
    x, dy = ((rows(s, M, n, FP32) * 2.0 ** low).to(dtype) for s, n in ((1, K), (2, N)))
    assert (x.float().abs() < torch.finfo(dtype).tiny).any() or dtype == FP32
    w, _, ad = layer(3, N, K, G, r, FP32)
    ad = cim.Adapters((ad.down * 2.0 ** up).to(dtype), (ad.up * 2.0 ** up).to(dtype), ad.scale)
    ids = numbers(4, M, G, "mixed")
    zero = torch.zeros_like(w)
    y, tol, h, dh = want_forward(x, zero, None, ad, ids, FP32)
    got, _, gh = cim.mxfp4_linear_adapters_nhwc(x, cim.mxfp4_quantize_nhwc(zero), None, ad, ids, out_dtype=FP32, save=True)
    ref.check(gh, h, dh + 2.0 ** -149, "h")
    ref.check(got, y, tol, "out")
    n = f64(ids).astype(np.int64)
    one = torch.ones((M, r), device="cuda")
    _, ddown, dup = cim.mxfp4_linear_adapters_bwd_nhwc(dy, torch.ones((M, K), device="cuda"), None, ad, ids, one)
    t, dt = kept.through(f64(dy), f64(ad.up), n)
    ref.check(ddown, *kept.grads(t, dt, np.ones((M, K)), f64(ad.scale), n), "ddown")
