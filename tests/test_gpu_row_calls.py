"""The row operators' calls from torch on the GPU: memory and streams."""
import pytest
import torch

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
