"""examples/channel_mixer.py: the operators together, as training and serving use them."""
import os
import sys

import numpy as np
import pytest
import torch

import row_reference as ref
from gpu_harness import need_gpu
from row_reference import f64

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import channel_mixer as cm  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def test_training_lowers_the_loss():
    _, losses = cm.train(steps=60)
    assert np.isfinite(losses).all()
    assert sum(losses[-5:]) < 0.5 * sum(losses[:5])


def test_served_block_equals_the_trained_one():
    """The fused norm quantises from fp32, the training path from bf16: values next to a border of the 4-bit grid take the
    neighbouring one, half a step of 4 bits apart at most, so outputs differ by a few of those among C terms."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    p = cm.block(gen)
    x = torch.randn(2, 9, 7, cm.C, generator=gen, device="cuda").bfloat16()
    h = cm.cim.conv2d_nhwc(x, p["conv"].bfloat16(), pad=1)
    n = cm.cim.layer_norm_nhwc(h, p["gamma"], p["beta"], cm.EPS, out_dtype=torch.float32)
    got = cm.Served(p)(x)
    assert got.shape == (2, 9, 7, cm.EXPAND)
    want, tol = ref.product(ref.mx_quantize(f64(n).reshape(-1, cm.C))[2], ref.mx_quantize(f64(p["w"]))[2], f64(p["b"]),
                            torch.bfloat16)
    ref.check(got.view(-1, cm.EXPAND), want, tol, "served block")


def test_gradients_follow_the_loss():
    """Along the gradient of beta and b, which enter the loss smoothly or nearly so, the loss falls at the gradient's rate."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    p = cm.block(gen)
    x = torch.randn(4, 14, 14, cm.C, generator=gen, device="cuda").bfloat16()
    want = torch.randn(4, 14, 14, cm.EXPAND, generator=gen, device="cuda")
    loss = lambda q: float((cm.forward(q, x)[0].double() - want.double()).square().sum())      # noqa: E731
    y, saved = cm.forward(p, x)
    g = cm.backward(p, x, saved, 2 * (y - want))
    # the loss is quadratic in b, so a central difference is exact up to fp32's roundings of y
    h = 1e-2
    d = g["b"] / g["b"].norm()
    up, down = (loss({**p, "b": p["b"] + s * h * d}) for s in (1, -1))
    slope, rate = (up - down) / (2 * h), float(g["b"].double().norm())
    assert abs(slope - rate) < 1e-3 * rate
