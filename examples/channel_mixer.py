"""Trains and serves a small channels-last block on one GPU:

    y = W q(norm(conv3x3(x))) + b

a 3x3 convolution, layer norm over the channels, and a pointwise (1x1)
convolution on 4-bit operands, with every gradient from the library.  The
data are random maps and the outputs of a fixed block of the same form.

    python examples/channel_mixer.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import convolution_implicit_gemm_fwd_amd as cim  # noqa: E402

C, EXPAND, EPS = 64, 256, 1e-5


def block(gen):
    """fp32 parameters: conv [C,3,3,C], gamma, beta [C], w [EXPAND,C], b [EXPAND]."""
    def normal(*shape, scale=1.0):
        return scale * torch.randn(*shape, generator=gen, device="cuda")

    return dict(conv=normal(C, 3, 3, C, scale=(9 * C) ** -0.5), gamma=1 + 0.1 * normal(C), beta=0.1 * normal(C),
                w=normal(EXPAND, C, scale=C ** -0.5), b=0.1 * normal(EXPAND))


def forward(p, x):
    """y (fp32) and what the backward pass needs."""
    h = cim.conv2d_nhwc(x, p["conv"].bfloat16(), pad=1)
    n, mean, rstd = cim.layer_norm_nhwc(h, p["gamma"], p["beta"], EPS, out_dtype=torch.bfloat16, stats=True)
    y = cim.mxfp4_linear_nhwc(n, cim.mxfp4_quantize_nhwc(p["w"]), p["b"], out_dtype=torch.float32)
    return y, (h, n, mean, rstd)


def backward(p, x, saved, dy):
    """The parameters' gradients."""
    h, n, mean, rstd = saved
    dn, dw, db = cim.mxfp4_linear_bwd_nhwc(dy, n, p["w"].to(n.dtype))
    dh, dgamma, dbeta = cim.layer_norm_bwd_nhwc(dn, h, p["gamma"], mean, rstd, dx_dtype=torch.bfloat16)
    dconv = cim.conv2d_bwd_weight_nhwc(x, dh, 3, 3, pad=1)
    return dict(conv=dconv, gamma=dgamma, beta=dbeta, w=dw, b=db)


class Served:
    """The block with its weights laid out once."""

    def __init__(self, p):
        self.p = p
        self.conv = p["conv"].bfloat16()
        self.w = cim.mxfp4_quantize_nhwc(p["w"])

    def __call__(self, x):
        h = cim.conv2d_nhwc(x, self.conv, pad=1)
        q = cim.layer_norm_mxfp4_nhwc(h, self.p["gamma"], self.p["beta"], EPS)
        return cim.mxfp4_linear_nhwc(q, self.w, self.p["b"], out_dtype=torch.bfloat16).view(*x.shape[:3], EXPAND)


def train(steps=60, rate=4.0, batch=8, size=14, seed=0):
    """(parameters, loss of each step, as a list of numbers)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    goal, p = block(gen), block(gen)
    losses = []
    for _ in range(steps):
        x = torch.randn(batch, size, size, C, generator=gen, device="cuda").bfloat16()
        want = forward(goal, x)[0]
        y, saved = forward(p, x)
        d = y - want
        losses.append(d.square().mean())
        # of the loss summed over channels, so that one rate fits every width
        g = backward(p, x, saved, (2.0 / d[..., 0].numel() * d).bfloat16())
        for k in p:
            p[k] -= rate / EXPAND * g[k]
    return p, [float(v) for v in losses]


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 200
    p, losses = train(steps)
    for k in range(0, steps, max(1, steps // 10)):
        print("step %4d  loss %.4f" % (k, losses[k]))
    print("step %4d  loss %.4f" % (steps - 1, losses[-1]))
    x = torch.randn(1, 14, 14, C, device="cuda").bfloat16()
    y, z = forward(p, x)[0], Served(p)(x)
    print("served block against the trained one: largest difference %.3f of %.3f"
          % (float((y - z).abs().max()), float(y.abs().max())))


if __name__ == "__main__":
    main()
