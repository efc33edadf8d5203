"""The row operators' calls from torch on the GPU: memory and streams."""
import pytest
import torch

import convolution_implicit_gemm_fwd_amd as cim
from gpu_harness import need_gpu
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
