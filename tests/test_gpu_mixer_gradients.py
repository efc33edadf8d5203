"""Every gradient of examples/channel_mixer.py's block against the chain rule in 64 bits, step by step on the maps that the
steps between them gave."""
import numpy as np
import pytest
import torch

import oracle
import row_reference as ref
from gpu_harness import need_gpu
from row_reference import U, f64
from test_gpu_channel_mixer import cm
from test_gpu_layer_norm import parts_chain

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def flat(t):
    return f64(t).reshape(-1, t.shape[-1])


def test_every_gradient_of_the_block(monkeypatch):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    p = cm.block(gen)
    x = torch.randn(3, 9, 11, cm.C, generator=gen, device="cuda").bfloat16()
    y, saved = cm.forward(p, x)
    dy = torch.randn(y.shape, generator=gen, device="cuda").bfloat16()
    h, n, mean, rstd = saved
    between = {}
    for name in ("mxfp4_linear_bwd_nhwc", "layer_norm_bwd_nhwc"):
        def step(*a, _f=getattr(cm.cim, name), _n=name, **k):
            between[_n] = _f(*a, **k)
            return between[_n]
        monkeypatch.setattr(cm.cim, name, step)
    g = cm.backward(p, x, saved, dy)
    dn, dh = between["mxfp4_linear_bwd_nhwc"][0], between["layer_norm_bwd_nhwc"][0]

    # the pointwise layer: y = Q(n) Q(w)^T + b, each product's operands in blocks along its sum
    d, w, m = flat(dy), f64(p["w"].bfloat16()), flat(dy).shape[0]
    q = lambda a: ref.mx_quantize(a)[2]      # noqa: E731
    ref.check(dn.view(-1, cm.C), *ref.product(q(d), q(w.T), None, BF16), "dn")
    ref.check(g["w"], *ref.product(q(d.T), q(flat(n).T), None, FP32), "w")
    ref.check(g["b"], d.sum(0), (-(-m // 128) + 128 + 16) * U * np.abs(d).sum(0), "b")
    # the norm of h
    want = ref.layer_norm_bwd(flat(dn), flat(h), f64(p["gamma"]), f64(mean).reshape(-1), f64(rstd).reshape(-1), BF16,
                              parts_chain(m))
    ref.check(dh.view(-1, cm.C), want[0], want[3], "dh")
    ref.check(g["gamma"], want[1], want[4], "gamma")
    ref.check(g["beta"], want[2], want[5], "beta")
    # the convolution: products of bf16 are exact in fp32, a sum has one term a pixel and at most as many partial sums
    dw, s = oracle.conv2d_bwd_weight(f64(x), f64(dh), 3, 3, 1, 1, 1)
    ref.check(g["conv"], dw, 2 * m * U * s + 1e-40, "conv")
    assert set(g) == set(p)
