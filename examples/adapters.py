"""Fine-tunes several users' low-rank adapters on one frozen layer in 4 bits and
serves their requests together, on one GPU:

    y = W q(norm(x)) + b + s_g up_g^T (down_g norm(x)),   g the user of the row

Each step's batch holds rows of all users.  What the gradients need is kept in
8 bits: the normalised rows for the norm's, the layer's input for the
adapters'.  The data are random rows and the outputs of the same layer with
other adapters.

    python examples/adapters.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import convolution_implicit_gemm_fwd_amd as cim  # noqa: E402

K, N, RANK, USERS, EPS = 256, 512, 8, 4, 1e-5


class Base:
    """The frozen layer: its weights in 4 bits both ways (forward, and backward along N)."""

    def __init__(self, gen):
        w = torch.randn(N, K, generator=gen, device="cuda") * K ** -0.5
        self.w, self.wt = cim.mxfp4_quantize_nhwc(w), cim.mxfp4_quantize_nhwc(w, transpose=True)
        self.bias = 0.1 * torch.randn(N, generator=gen, device="cuda")


def users(gen, up=1.0):
    """fp32 parameters: gamma and beta [K], down [USERS, RANK, K], up [USERS, RANK, N]."""
    def normal(*shape, scale=1.0):
        return scale * torch.randn(*shape, generator=gen, device="cuda")

    return dict(gamma=1 + 0.1 * normal(K), beta=0.1 * normal(K), down=normal(USERS, RANK, K, scale=K ** -0.5),
                up=normal(USERS, RANK, N, scale=up * RANK ** -0.5))


def adapters(p):
    return cim.Adapters(p["down"].bfloat16(), p["up"].bfloat16(), torch.full((USERS,), 0.5, device="cuda"))


def forward(base, p, x, ids):
    """y (fp32) and what the backward pass needs."""
    n, kept_n, rstd = cim.layer_norm_mxint8_nhwc(x, p["gamma"], p["beta"], EPS, out_dtype=torch.bfloat16)
    y, kept, h = cim.mxfp4_linear_adapters_nhwc(n, base.w, base.bias, adapters(p), ids, out_dtype=torch.float32, save=True)
    return y, (kept_n, rstd, kept, h)


def backward(base, p, ids, saved, dy):
    """The parameters' gradients."""
    kept_n, rstd, kept, h = saved
    dn, ddown, dup = cim.mxfp4_linear_adapters_bwd_nhwc(dy, kept, base.wt, adapters(p), ids, h)
    _, dgamma, dbeta = cim.layer_norm_bwd_mxint8_nhwc(dn, kept_n, p["gamma"], rstd)
    return dict(gamma=dgamma, beta=dbeta, down=ddown, up=dup)


class Served:
    """The layer with every user's adapter at hand."""

    def __init__(self, base, p):
        self.base, self.p, self.adapters = base, p, adapters(p)

    def __call__(self, x, ids):
        n = cim.layer_norm_nhwc(x, self.p["gamma"], self.p["beta"], EPS, out_dtype=torch.bfloat16)
        return cim.mxfp4_linear_adapters_nhwc(n, self.base.w, self.base.bias, self.adapters, ids)


def train(steps=40, rate=20.0, rows=512, seed=0):
    """(base, parameters, loss of each step, as a list of numbers)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    base = Base(gen)
    goal, p = users(gen), users(gen, up=0.0)
    losses = []
    for _ in range(steps):
        x = torch.randn(rows, K, generator=gen, device="cuda").bfloat16()
        ids = torch.randint(-1, USERS, (rows,), generator=gen, device="cuda").int()      # -1: the layer alone
        want = forward(base, goal, x, ids)[0]
        y, saved = forward(base, p, x, ids)
        d = y - want
        losses.append(d.square().mean())
        g = backward(base, p, ids, saved, (2.0 / rows * d).bfloat16())
        for k in p:
            p[k] -= rate / N * g[k] if k in ("gamma", "beta") else rate * USERS / N * g[k]
    return base, p, [float(v) for v in losses]


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 200
    base, p, losses = train(steps)
    for k in range(0, steps, max(1, steps // 10)):
        print("step %4d  loss %.4f" % (k, losses[k]))
    print("step %4d  loss %.4f" % (steps - 1, losses[-1]))
    served = Served(base, p)
    x = torch.randn(5, K, device="cuda").bfloat16()
    ids = torch.tensor([2, 0, -1, 3, 2], dtype=torch.int32, device="cuda")
    y, z = forward(base, p, x, ids)[0], served(x, ids)
    print("served requests against the trained layer: largest difference %.3f of %.3f"
          % (float((y - z).abs().max()), float(y.abs().max())))


if __name__ == "__main__":
    main()
