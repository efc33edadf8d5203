"""The convolution's torch wrappers on another stream, on the CPU: stand-ins for the library's calls and for torch's
streams, and tensors of host memory that pass for device tensors (test_row_wrappers_host.py)."""
import contextlib

import pytest
import torch

import convolution_implicit_gemm_fwd_amd as cim
from test_row_wrappers_host import HOME, SIDE, Dev, Stream, dev


@pytest.fixture
def machine(monkeypatch):
    class Machine:
        current, made, streams = HOME, {}, []

    m = Machine()
    m.made, m.streams, Dev.recorded = {}, [], []

    def set_stream(s):
        m.current = s.cuda_stream

    @contextlib.contextmanager
    def under(s):
        before, m.current = m.current, s.cuda_stream
        yield
        m.current = before

    def empty(*a, _empty=torch.empty, **k):
        t = dev(_empty(*a, **k))
        m.made[t.data_ptr()] = m.current
        return t

    def entry(*args):
        m.streams.append(args[-1])
        return 0

    for name, f in dict(set_stream=set_stream, stream=under, ExternalStream=Stream, device=contextlib.nullcontext,
                        current_stream=lambda device=None: Stream(m.current)).items():
        monkeypatch.setattr(torch.cuda, name, f)
    monkeypatch.setattr(torch, "empty", empty)
    for name in ("conv2d_fwd", "conv2d_bwd_data", "conv2d_bwd_weight", "conv2d_fwd_nchw"):
        monkeypatch.setattr(cim, name, entry)
    monkeypatch.setattr(cim, "conv2d_bwd_weight_workspace", lambda *a: (0, 4096))
    monkeypatch.setattr(cim, "conv2d_fwd_nchw_workspace", lambda *a: (0, 4096))
    return m


def calls():
    x, w, dy = dev(torch.ones(2, 8, 8, 64)), dev(torch.ones(32, 3, 3, 64)), dev(torch.ones(2, 8, 8, 32))
    return [lambda s: cim.conv2d_nhwc(x, w, None, 1, 1, stream=s),
            lambda s: cim.conv2d_bwd_data_nhwc(dy, w, 8, 8, 1, 1, stream=s),
            lambda s: cim.conv2d_bwd_weight_nhwc(x, dy, 3, 3, 1, 1, stream=s),
            lambda s: cim.conv2d_nchw(dev(torch.ones(2, 64, 8, 8)), dev(torch.ones(32, 64, 3, 3)), None, 1, 1, stream=s)]


@pytest.mark.parametrize("k", range(4))
def test_buffers_of_another_stream_are_its_own(machine, k):
    """A block of the current stream's pool may still be in use by work that is queued there: what a call on another
    stream writes comes from that stream's pool, and the result is not reused before the current stream is past it."""
    call = calls()[k]
    out = call(SIDE)
    assert machine.streams == [SIDE] and machine.current == HOME
    assert machine.made and set(machine.made.values()) == {SIDE}
    assert (out.data_ptr(), HOME) in Dev.recorded
    machine.made.clear()
    Dev.recorded.clear()
    for s in (None, HOME):
        call(s)
        assert machine.streams[-1] == HOME and set(machine.made.values()) == {HOME} and not Dev.recorded
