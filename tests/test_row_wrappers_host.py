"""What the row operators' torch wrappers hand to the C library, on the CPU: a stand-in for the library records the
addresses it gets, tensors of host memory pass for device tensors, and a stand-in for torch's streams tells which one is
current."""
import ctypes
import gc
import types

import pytest
import torch

from convolution_implicit_gemm_fwd_amd import abi
from convolution_implicit_gemm_fwd_amd import rows as R

HOME, SIDE = 0, 0x5000      # stream handles


class Dev(torch.Tensor):
    """A host tensor that passes for a device tensor."""
    is_cuda = property(lambda self: True)

    def record_stream(self, stream):
        Dev.recorded.append((self.data_ptr(), stream.cuda_stream))


def dev(t):
    return t.as_subclass(Dev)


class Stream:
    def __init__(self, cuda_stream, device=None):
        self.cuda_stream = cuda_stream


class Machine:
    """Streams, allocations and library calls as the wrappers make them."""

    def __init__(self, monkeypatch):
        self.current, self.made, self.calls = HOME, {}, []
        Dev.recorded = []
        machine = self

        def set_stream(stream):
            machine.current = stream.cuda_stream

        def made(t):
            t = dev(t)
            self.made[t.data_ptr()] = self.current
            return t

        cuda = types.SimpleNamespace(set_stream=set_stream, ExternalStream=Stream, device=None,
                                     current_stream=lambda device=None: Stream(self.current))
        R._torch or R._setup()
        for name, value in dict(
                _torch=types.SimpleNamespace(cuda=cuda, empty_like=lambda t, dtype=None: made(torch.empty_like(t, dtype=dtype)),
                                             Tensor=torch.Tensor, bfloat16=torch.bfloat16),
                _empty=lambda *a, **k: made(torch.empty(*a, **k)), _device=lambda: None, _stream=lambda index: self.current,
                _fast=types.SimpleNamespace(**{n: lambda *a: None for n in (
                    "layer_norm", "layer_norm_mxfp4", "layer_norm_bwd", "quantize", "dequantize", "linear", "linear_bwd")}),
                _lib=types.SimpleNamespace(**{n: self.entry(n) for n in (
                    "layer_norm_fwd", "layer_norm_fwd_mxfp4", "layer_norm_bwd", "mxfp4_quantize", "mxfp4_dequantize",
                    "mxfp4_linear_fwd", "mxfp4_linear_bwd")})).items():
            monkeypatch.setattr(R, name, value)

    def entry(self, name):
        def call(*args):
            self.calls.append((name, args))
            return self.check(name, args) or 0
        return call

    def check(self, name, args):
        pass


@pytest.fixture
def machine(monkeypatch):
    return Machine(monkeypatch)


def calls():
    x, w, dy = dev(torch.ones(300, 256)), dev(torch.ones(128, 256)), dev(torch.ones(300, 128))
    mean, rstd = dev(torch.ones(300)), dev(torch.ones(300))
    q = R.Mxfp4Tensor(dev(torch.zeros(128, 128, dtype=torch.uint8)), dev(torch.zeros(2, 128, 4, dtype=torch.uint8)), 128, 256)
    return [lambda **s: R.layer_norm_nhwc(x, stats=True, **s), lambda **s: R.layer_norm_mxfp4_nhwc(x, **s),
            lambda **s: R.layer_norm_bwd_nhwc(x, x, None, mean, rstd, **s), lambda **s: R.mxfp4_quantize_nhwc(x, **s),
            lambda **s: R.mxfp4_dequantize_nhwc(q, torch.float32, **s), lambda **s: R.mxfp4_linear_nhwc(x, q, **s),
            lambda **s: R.mxfp4_linear_nhwc(q, q, **s), lambda **s: R.mxfp4_linear_bwd_nhwc(dy, x, w, **s)]


def test_packed_rows_come_with_statistics(machine):
    x = dev(torch.ones(3, 5, 64))
    q, mean, rstd = R.layer_norm_mxfp4_nhwc(x, stats=True, stream=SIDE)
    assert isinstance(q, R.Mxfp4Tensor) and mean.shape == rstd.shape == (3, 5)
    args = machine.calls[-1][1]
    assert args[8:13] == (q.codes.data_ptr(), q.scales.data_ptr(), mean.data_ptr(), rstd.data_ptr(), SIDE)
    assert {(t.data_ptr(), HOME) for t in (q.codes, q.scales, mean, rstd)} <= set(Dev.recorded)
    q = R.layer_norm_mxfp4_nhwc(x)
    assert isinstance(q, R.Mxfp4Tensor) and machine.calls[-1][1][10:12] == (None, None)


def tensors(r):
    return [r] if isinstance(r, torch.Tensor) else [t for v in r if not isinstance(v, int) for t in tensors(v)]


@pytest.mark.parametrize("k", range(8))
def test_buffers_of_another_stream_are_its_own(machine, k):
    """A block of the current stream's pool may still be in use by work that is queued there: what a call on another
    stream writes comes from that stream's pool, and the results are not reused before the current stream is past them."""
    call = calls()[k]
    out = tensors(call(stream=SIDE))
    assert machine.calls[-1][1][-1] == SIDE
    assert machine.made and set(machine.made.values()) == {SIDE}
    assert {(t.data_ptr(), HOME) for t in out} <= set(Dev.recorded)
    assert machine.current == HOME
    machine.made.clear()
    Dev.recorded.clear()
    for s in (None, HOME):
        call(stream=s)
        assert machine.calls[-1][1][-1] == HOME and set(machine.made.values()) == {HOME} and not Dev.recorded


def held(address):
    """Whether a tensor that is still held covers the address."""
    return any(isinstance(t, torch.Tensor) and t.data_ptr() <= address < t.data_ptr() + max(1, t.numel() * t.element_size())
               for t in gc.get_objects() if isinstance(t, torch.Tensor) and t.device.type == "cpu")


def floats(address, n):
    return list((ctypes.c_float * n).from_address(address))


@pytest.mark.parametrize("stream", [None, SIDE])
@pytest.mark.parametrize("lay", [lambda t: t, lambda t: t.t().contiguous().t(), lambda t: torch.stack((t, t), -1)[..., 1],
                                 lambda t: torch.cat((t, t), 1)[:, :t.shape[1]],
                                 lambda t: torch.stack((t.reshape(-1), t.reshape(-1)), -1)[:, 0]],
                         ids=["contiguous", "transposed", "every other", "narrowed", "strided vector"])
def test_statistics_of_any_layout_are_there_when_the_kernel_reads_them(machine, lay, stream):
    """The kernel gets the statistics themselves, or copies that are held until after the call."""
    n, h, c = 5, 7, 16
    mean, rstd = torch.arange(35.).view(n, h), 100 + torch.arange(35.).view(n, h)
    x = dev(torch.ones(n, h, c))
    seen = []

    def check(name, args):
        m, r = args[5], args[6]
        assert held(m) and held(r), "freed statistics"
        assert m != r and floats(m, 35) == mean.view(-1).tolist() and floats(r, 35) == rstd.view(-1).tolist()
        others = [args[k] for k in (0, 2, 13, 14, 15, 16)]
        assert m not in others and r not in others
        seen.append(machine.current)

    machine.check = check
    R.layer_norm_bwd_nhwc(x, x, None, dev(lay(mean)), dev(lay(rstd)), stream=stream)
    assert seen == [stream or HOME]


def far(*shape, dtype=torch.bfloat16):
    """A tensor of that shape without memory."""
    return dev(torch.empty(*shape, dtype=dtype, device="meta"))


MANY = (1 << 32) + 5      # 5 in 32 bits


@pytest.mark.parametrize("call", [
    lambda: R.layer_norm_nhwc(far(1, MANY)), lambda: R.layer_norm_mxfp4_nhwc(far(3, MANY)),
    lambda: R.layer_norm_bwd_nhwc(far(1, MANY), far(1, MANY), None, far(1, dtype=torch.float32), far(1, dtype=torch.float32)),
    lambda: R.mxfp4_quantize_nhwc(far(MANY, 32)), lambda: R.mxfp4_quantize_nhwc(far(MANY, 32), transpose=True),
    lambda: R.mxfp4_quantize_nhwc(far(1, MANY)), lambda: R.mxfp4_quantize_nhwc(far(1 << 31, 3)),
    lambda: R.mxfp4_dequantize_nhwc(packed(MANY, 32), torch.bfloat16),
    lambda: R.mxfp4_dequantize_nhwc(packed(2, MANY), torch.bfloat16),
    lambda: R.mxfp4_linear_nhwc(far(MANY, 32), packed(8, 32)), lambda: R.mxfp4_linear_nhwc(packed(MANY, 32), packed(8, 32)),
    lambda: R.mxfp4_linear_nhwc(far(8, 32), packed(MANY, 32)),
    lambda: R.mxfp4_linear_bwd_nhwc(far(MANY, 8), far(MANY, 32), far(8, 32)),
    lambda: R.mxfp4_linear_bwd_nhwc(far(4, MANY), far(4, 32), far(MANY, 32))], ids=range(14))
def test_sizes_past_the_library_s_32_bits_are_refused(machine, call):
    """They would reach the library as their lower 32 bits."""
    with pytest.raises(RuntimeError, match="status %d" % abi.CONVIMG_ERR_RANGE):
        call()
    assert not machine.calls


def packed(rows, cols):
    nb = -(-cols // 32)
    return R.Mxfp4Tensor(far(rows, nb * 16, dtype=torch.uint8), far(-(-nb // 4), rows, 4, dtype=torch.uint8), rows, cols)


def test_a_missing_torch_module_names_the_build(monkeypatch):
    import sys

    import convolution_implicit_gemm_fwd_amd as package

    monkeypatch.setattr(R, "_torch", None)
    monkeypatch.delattr(package, "_rows", raising=False)
    monkeypatch.setitem(sys.modules, package.__name__ + "._rows", None)
    with pytest.raises(abi.LibraryMissing, match="convolution_implicit_gemm_fwd_amd.build"):
        R.layer_norm_nhwc(torch.zeros(2, 8))
