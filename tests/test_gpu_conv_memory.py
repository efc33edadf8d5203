"""The convolution's torch wrappers on another stream, on the GPU: memory that queued work still uses."""
import pytest
import torch

import convolution_implicit_gemm_fwd_amd as cim
from gpu_harness import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def calls():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    t = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()      # noqa: E731
    x, w, dy = t(2, 16, 16, 64), t(96, 3, 3, 64), t(2, 16, 16, 96)
    xc, wc = x.permute(0, 3, 1, 2).contiguous(), w.permute(0, 3, 1, 2).contiguous()
    return [lambda **s: cim.conv2d_nhwc(x, w, pad=1, **s), lambda **s: cim.conv2d_bwd_data_nhwc(dy, w, 16, 16, pad=1, **s),
            lambda **s: cim.conv2d_bwd_weight_nhwc(x, dy, 3, 3, pad=1, **s), lambda **s: cim.conv2d_nchw(xc, wc, pad=1, **s)]


def test_memory_in_use_on_the_current_stream_is_left_alone():
    """Blocks that are free again while work queued on the current stream still reads them are not what a call on
    another stream writes to."""
    for k, call in enumerate(calls()):
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
        assert torch.equal(got, want), "call %d" % k
