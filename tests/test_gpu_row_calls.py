"""The row operators' calls from torch on the GPU: memory and streams."""
import pytest
import torch

import convolution_implicit_gemm_fwd_amd as cim
import row_reference as ref
from gpu_harness import need_gpu
from row_reference import f64
from test_gpu_layer_norm import EPS, params, parts_chain
from test_gpu_layer_norm import rows as norm_rows
from test_gpu_mxfp4 import side_stream_cases

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def test_memory_in_use_on_the_current_stream_is_left_alone():
    """Blocks that are free again while work queued on the current stream still reads them are not what a call on
    another stream writes to."""
    for k, call in enumerate(side_stream_cases()):
        want = call()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        kept = []
        for b in range(9, 21):
            block = torch.full((1 << b,), b, dtype=torch.uint8, device="cuda")
            kept.append(block.clone())
            del block
        got = call(stream=side.cuda_stream)
        torch.cuda.synchronize()
        assert all(bool((t == b).all()) for b, t in zip(range(9, 21), kept)), "call %d" % k
        for p, q in zip(got, want):
            assert torch.equal(p, q), "call %d" % k


@pytest.mark.parametrize("lay", [lambda t: t.transpose(0, 1).contiguous().transpose(0, 1), lambda t: t.repeat(1, 2)[:, :t.shape[1]],
                                 lambda t: torch.stack((t, t + 1), -1)[..., 0],
                                 lambda t: torch.stack((t.reshape(-1), t.reshape(-1) + 1), -1)[:, 0]],
                         ids=["transposed", "narrowed", "every other", "strided vector"])
def test_statistics_of_any_layout(lay):
    x, dy = torch.randn(2, 40, 50, 96, device="cuda").bfloat16().unbind(0)
    gamma = torch.rand(96, device="cuda") + 0.5
    _, mean, rstd = cim.layer_norm_nhwc(x, stats=True)
    want = cim.layer_norm_bwd_nhwc(dy, x, gamma, mean, rstd)
    m, r = lay(mean), lay(rstd)
    assert not m.is_contiguous() and not r.is_contiguous()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side.cuda_stream):
        for _ in range(3):
            got = cim.layer_norm_bwd_nhwc(dy, x, gamma, m, r, stream=stream)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("n,cols", [(1, 7), (70, 64), (9, 100), (300, 513), (2, 4100), (2, 8200)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_packed_rows_with_the_statistics_for_the_gradient(n, cols, dtype):
    """The rows are those of the call without statistics, and the statistics serve the gradient."""
    x, (g, b) = norm_rows(cols, n, cols, dtype), params(cols, cols)
    q, mean, rstd = cim.layer_norm_mxfp4_nhwc(x, g, b, EPS, stats=True)
    p = cim.layer_norm_mxfp4_nhwc(x, g, b, EPS)
    assert torch.equal(q.codes, p.codes) and torch.equal(q.scales, p.scales) and q[2:] == p[2:]
    _, m, r, _, dm, dr = ref.layer_norm(f64(x), f64(g), f64(b), EPS, torch.float32)
    ref.check(mean, m, dm, "mean")
    ref.check(rstd, r, dr, "rstd")
    dy = norm_rows(cols + 1, n, cols, dtype, scale=0.1, mean=0)
    dx, dg, db = cim.layer_norm_bwd_nhwc(dy, x, g, mean, rstd, dx_dtype=torch.float32)
    w = ref.layer_norm_bwd(f64(dy), f64(x), f64(g), f64(mean), f64(rstd), torch.float32, parts_chain(n))
    for got, want, tol, what in ((dx, w[0], w[3], "dx"), (dg, w[1], w[4], "dgamma"), (db, w[2], w[5], "dbeta")):
        ref.check(got, want, tol, what)
