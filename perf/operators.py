"""What is measured of the row operators: layer normalisation and its
gradient, microscaled 4-bit quantisation (MXFP4), the product of quantised
rows and its gradient.

Each case is one pass through one operator, on channels-last data: a row is
one token, or one pixel of an NHWC map, and its columns are the channels.
``run`` computes the plain form in 32 bits with elementary torch operations,
or, with ``own`` set, calls the package.

MXFP4: a block of 32 consecutive values along the contracted axis shares a
scale 2^(s - 127), s = clamp(floor(log2 max|x|) - 2 + 127, 0, 254); a value is
x / scale rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the
even code, larger values to 6) with its sign.  Packed: codes [rows][Kp / 2],
two a byte, the even column in the low half, Kp the columns rounded up to 32;
scales [ceil(Kp / 128)][rows][4], one byte a block.
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token before its projection: latency
        dict(name="norm, one token", op="norm", rows=1, cols=4096, dtype="bf16", out="bf16", pad=0, stats=False),
        # a convolution's fp32 map, 16 x 56 x 56 x 64, normalised for a bf16 layer, statistics kept for training
        dict(name="norm, 56x56x64 map", op="norm", rows=50176, cols=64, dtype="fp32", out="bf16", pad=0, stats=True),
        # the gradient on a 4 x 128 x 128 x 128 map
        dict(name="norm bwd, 128x128x128 map", op="norm_bwd", rows=65536, cols=128, dtype="bf16", grad="fp32", pad=0),
        # the gradient over a long training batch
        dict(name="norm bwd, 16384 tokens", op="norm_bwd", rows=16384, cols=4096, dtype="bf16", grad="bf16", pad=0),
        # quantise and restore rows of an odd width inside a wider buffer (calibration of a layer)
        dict(name="quantise, ragged rows", op="quantise", rows=1237, cols=2013, dtype="fp16", pad=35, t=False),
        # the same down the columns of a large activation, as the weight's gradient contracts it
        dict(name="quantise, down columns", op="quantise", rows=8192, cols=8192, dtype="bf16", pad=0, t=True),
        # one token through a projection
        dict(name="linear, one token", op="linear", M=1, N=4096, K=4096, dtype="bf16", out="bf16", norm=False),
        # a small serving batch, ragged
        dict(name="linear, 37 tokens", op="linear", M=37, N=8000, K=4096, dtype="bf16", out="bf16", norm=False),
        # the pointwise expansion after the norm on a 16 x 14 x 14 x 512 map; 16-bit out, as the norm's last bit
        # decides which of two grid values a few activations take
        dict(name="norm + linear, 14x14x512 map", op="linear", M=3136, N=2048, K=512, dtype="fp32", out="bf16", norm=True),
        # a long prompt
        dict(name="linear, 8192 tokens", op="linear", M=8192, N=8192, K=8192, dtype="bf16", out="bf16", norm=False),
        # the gradient of a pointwise layer on an odd number of pixels
        dict(name="linear bwd, 1000 pixels", op="linear_bwd", M=1000, N=512, K=130, dtype="fp32", grad="fp32"),
        # the gradient over a training batch
        dict(name="linear bwd, 8192 tokens", op="linear_bwd", M=8192, N=4096, K=4096, dtype="bf16", grad="bf16"),
    ]


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    def kind():
        return rng.choice(sorted(TYPES))

    op = rng.choice(["norm", "norm_bwd", "quantise", "linear", "linear_bwd"])
    pad = rng.choice([0, 0, rng.randrange(1, 64)])
    if op in ("norm", "norm_bwd", "quantise"):
        cols = size(16, 8192)
        rows = size(1, min(65536, 2 ** 26 // cols))
        c = dict(op=op, rows=rows, cols=cols, dtype=kind(), pad=pad)
        if op == "norm":
            c.update(out=kind(), stats=rng.random() < 0.5)
        elif op == "norm_bwd":
            c.update(grad=kind())
        else:
            c.update(t=rng.random() < 0.5)
        return c
    if op == "linear":
        norm = rng.random() < 0.3
        return dict(op=op, M=size(1, 8192), N=size(16, 8192), K=size(16, 8192), dtype=kind(),
                    out=rng.choice(["bf16", "fp16"]) if norm else kind(), norm=norm)
    return dict(op=op, M=size(16, 8192), N=size(16, 4096), K=size(16, 4096), dtype=kind(), grad=kind())


# ---- MXFP4 in plain torch ------------------------------------------------

def _values():
    v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(v + [-a for a in v], device="cuda")


def _blocks(x):
    """fp32 [rows, blocks, 32], zeros past the last column."""
    k = x.shape[1]
    kp = -(-k // 32) * 32
    y = torch.zeros(x.shape[0], kp, device=x.device)
    y[:, :k] = x
    return y.view(x.shape[0], kp // 32, 32)


def _scale_bytes(b):
    """One byte a block: the exponent field of the largest magnitude, less 2."""
    top = b.abs().amax(-1).view(torch.int32) >> 23
    return (top - 2).clamp_min(0)


def _power(s):
    """2^(s - 127) in fp32 for whole s of 0 to 254."""
    return torch.where(s > 0, s << 23, torch.full_like(s, 1 << 22)).to(torch.int32).view(torch.float32)


def _rounded(b, s):
    """The blocks over their scales, rounded to the grid."""
    v = b * _power(254 - s).unsqueeze(-1)
    a = v.abs()
    r = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return torch.copysign(r.clamp_max(6), v)


def _fake(x):
    """fp32 [rows, K]: what the quantised rows stand for."""
    b = _blocks(x)
    s = _scale_bytes(b)
    return (_rounded(b, s) * _power(s).unsqueeze(-1)).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _packed(w):
    """codes and scales of fp32 rows, as a program keeps its weights."""
    b = _blocks(w)
    n, nb, _ = b.shape
    s = _scale_bytes(b)
    r = _rounded(b, s)
    a = r.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(r).to(torch.uint8) << 3)).view(n, nb * 16, 2)
    quads = -(-nb // 4)
    scales = torch.zeros(n, quads * 4, dtype=torch.uint8, device=w.device)
    scales[:, :nb] = s.to(torch.uint8)
    return code[:, :, 0] | (code[:, :, 1] << 4), scales.view(n, quads, 4).permute(1, 0, 2).contiguous()


def _unpacked(codes, scales, k):
    n = codes.shape[0]
    q = torch.stack((codes & 15, codes >> 4), -1).to(torch.int32).reshape(n, -1, 32)
    s = scales.permute(1, 0, 2).reshape(n, -1)[:, :q.shape[1]].to(torch.int32)
    return (_values()[q] * _power(s).unsqueeze(-1)).reshape(n, -1)[:, :k]


# ---- inputs ---------------------------------------------------------------

def _rows(gen, rows, cols, dtype, pad=0):
    """Activations: normal rows with an offset, some channels far larger."""
    x = torch.randn(rows, cols + pad, generator=gen, device="cuda")
    loud = torch.where(torch.rand(cols + pad, generator=gen, device="cuda") < 0.02, 8.0, 1.0)
    x = x * loud + 0.3 * torch.randn(rows, 1, generator=gen, device="cuda") + 0.1
    return x.to(TYPES[dtype])[:, :cols]


def _grads(gen, rows, cols, dtype, pad=0):
    """Output gradients: normal, each row of its own size."""
    g = torch.randn(rows, cols + pad, generator=gen, device="cuda")
    g = g * torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device="cuda"))
    return (g * 0.05).to(TYPES[dtype])[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op in ("norm", "norm_bwd", "quantise"):
        s["x"] = _rows(gen, case["rows"], case["cols"], case["dtype"], case["pad"])
    if op in ("norm", "norm_bwd"):
        s["gamma"] = 1 + 0.1 * torch.randn(case["cols"], generator=gen, device="cuda")
        s["beta"] = 0.1 * torch.randn(case["cols"], generator=gen, device="cuda")
    if op == "norm_bwd":
        s["dy"] = _grads(gen, case["rows"], case["cols"], case["grad"], case["pad"])
        x = s["x"].float()
        m = x.mean(-1)
        s["mean"] = m
        s["rstd"] = torch.rsqrt((x - m[:, None]).square().mean(-1) + EPS)
    if op in ("linear", "linear_bwd"):
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _rows(gen, M, K, case["dtype"])
        w = torch.randn(N, K, generator=gen, device="cuda") / math.sqrt(K)
        if op == "linear":
            s["codes"], s["scales"] = _packed(w)
            s["bias"] = 0.1 * torch.randn(N, generator=gen, device="cuda")
            if case["norm"]:
                s["gamma"] = 1 + 0.1 * torch.randn(K, generator=gen, device="cuda")
                s["beta"] = 0.1 * torch.randn(K, generator=gen, device="cuda")
        else:
            s["w"] = w.to(TYPES[case["dtype"]])
            s["dy"] = _grads(gen, M, N, case["grad"])
    return s


# ---- one pass -------------------------------------------------------------

def _norm(x, gamma, beta):
    x = x.float()
    mean = x.mean(-1)
    c = x - mean[:, None]
    rstd = torch.rsqrt(c.square().mean(-1) + EPS)
    return c * rstd[:, None] * gamma + beta, mean, rstd


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    op = c["op"]
    if op == "norm":
        y, mean, rstd = _norm(state["x"], state["gamma"], state["beta"])
        y = y.to(TYPES[c["out"]])
        return (y, mean, rstd) if c["stats"] else y
    if op == "norm_bwd":
        dy = state["dy"].float()
        xhat = (state["x"].float() - state["mean"][:, None]) * state["rstd"][:, None]
        g = dy * state["gamma"]
        dx = state["rstd"][:, None] * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
        return dx.to(state["x"].dtype), (dy * xhat).sum(0), dy.sum(0)
    if op == "quantise":
        x = state["x"].float()
        return _fake(x.t() if c["t"] else x).to(state["x"].dtype)
    if op == "linear":
        x = state["x"].float()
        if c["norm"]:
            x = _norm(x, state["gamma"], state["beta"])[0]
        y = torch.matmul(_fake(x), _unpacked(state["codes"], state["scales"], c["K"]).t()) + state["bias"]
        return y.to(TYPES[c["out"]])
    dy, x, w = state["dy"].float(), state["x"].float(), state["w"].float()
    dx = torch.matmul(_fake(dy), _fake(w.t()).t())
    dw = torch.matmul(_fake(dy.t()), _fake(x.t()).t())
    return dx.to(state["x"].dtype), dw, dy.sum(0)


def _run_own(state):
    import convolution_implicit_gemm_fwd_amd as cim

    c = state["case"]
    op = c["op"]
    if op == "norm":
        return cim.layer_norm_nhwc(state["x"], state["gamma"], state["beta"], eps=EPS, out_dtype=TYPES[c["out"]],
                                   stats=c["stats"])
    if op == "norm_bwd":
        return cim.layer_norm_bwd_nhwc(state["dy"], state["x"], state["gamma"], state["mean"], state["rstd"])
    if op == "quantise":
        q = cim.mxfp4_quantize_nhwc(state["x"], transpose=c["t"])
        return cim.mxfp4_dequantize_nhwc(q, state["x"].dtype)
    if op == "linear":
        w = cim.Mxfp4Tensor(state["codes"], state["scales"], c["N"], c["K"])
        x = state["x"]
        if c["norm"]:
            x = cim.layer_norm_mxfp4_nhwc(x, state["gamma"], state["beta"], eps=EPS)
        return cim.mxfp4_linear_nhwc(x, w, state["bias"], out_dtype=TYPES[c["out"]])
    return cim.mxfp4_linear_bwd_nhwc(state["dy"], state["x"], state["w"])


# ---- what a pass cannot do without ---------------------------------------

def work(case):
    def b(t):
        return TYPES[t].itemsize

    def mx(rows, cols):
        blocks = rows * -(-cols // 32)
        return blocks * 17

    op = case["op"]
    if op in ("norm", "norm_bwd", "quantise"):
        r, k = case["rows"], case["cols"]
        e = r * k
        if op == "norm":
            return dict(bytes=e * (b(case["dtype"]) + b(case["out"])) + 8 * k + (8 * r if case["stats"] else 0),
                        flops=8 * e)
        if op == "norm_bwd":
            return dict(bytes=e * (2 * b(case["dtype"]) + b(case["grad"])) + 12 * k + 8 * r, flops=14 * e)
        return dict(bytes=2 * e * b(case["dtype"]) + (mx(k, r) if case["t"] else mx(r, k)), flops=4 * e)
    M, N, K = case["M"], case["N"], case["K"]
    if op == "linear":
        return dict(bytes=M * K * b(case["dtype"]) + mx(N, K) + M * N * b(case["out"]) + 4 * N
                    + (8 * K if case["norm"] else 0), flops=2 * M * N * K)
    return dict(bytes=M * N * b(case["grad"]) + 2 * M * K * b(case["dtype"]) + N * K * (b(case["dtype"]) + 4) + 4 * N,
                flops=4 * M * N * K)


# ---- the definitions in 64 bits -------------------------------------------

def _exact_power(e):
    """2^e in fp64 for whole e, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_fake(x):
    """Along the last axis, by thresholds between neighbouring grid values."""
    n, k = x.shape
    pad = (-k) % 32
    b = torch.nn.functional.pad(x, (0, pad)).reshape(n, -1, 32)
    _, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = torch.where((b == 0).all(-1, keepdim=True), torch.full_like(e, -200), e - 3).clamp(-127, 127)
    unit = _exact_power(e)
    a = b.abs() / unit
    q = 0.5 * ((a > 0.25).double() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) \
        + (a > 2.5).double() + (a >= 3.5).double() + 2 * (a > 5).double()
    return (torch.sign(b) * q * unit).reshape(n, -1)[:, :k]


def _exact_weights(codes, scales, n, k):
    lo, hi = codes.long() % 16, codes.long() // 16
    q = torch.empty(n, 2 * codes.shape[1], dtype=torch.long, device=codes.device)
    q[:, 0::2], q[:, 1::2] = lo, hi
    e, m = (q % 8) // 2, (q % 2).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * _exact_power(e - 1))
    col = torch.arange(q.shape[1], device=codes.device)
    s = scales.long()[col // 128, :, (col // 32) % 4].t()
    return (torch.where(q >= 8, -mag, mag) * _exact_power(s - 127))[:, :k]


def _exact_norm(x, gamma, beta):
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    return (x - mean) / (var + EPS).sqrt() * gamma.double() + beta.double(), mean[:, 0], (var[:, 0] + EPS) ** -0.5


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    x = s["x"].double()
    if op == "norm":
        out = _exact_norm(x, s["gamma"], s["beta"])
        return out if case["stats"] else out[0]
    if op == "norm_bwd":
        dy, mean, rstd = s["dy"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
        n = (x - mean) * rstd
        h = dy * s["gamma"].double()
        k = x.shape[1]
        return rstd / k * (k * h - h.sum(-1, keepdim=True) - n * (h * n).sum(-1, keepdim=True)), \
            (dy * n).sum(0), dy.sum(0)
    if op == "quantise":
        return _exact_fake(x.t().contiguous() if case["t"] else x)
    if op == "linear":
        if case["norm"]:
            x = _exact_norm(x, s["gamma"], s["beta"])[0]
        w = _exact_weights(s["codes"], s["scales"], case["N"], case["K"])
        return _exact_fake(x) @ w.t().contiguous() + s["bias"].double()
    dy, w = s["dy"].double(), s["w"].double()
    dyt, xt, wt = (t.t().contiguous() for t in (dy, x, w))
    return _exact_fake(dy) @ _exact_fake(wt).t().contiguous(), _exact_fake(dyt) @ _exact_fake(xt).t().contiguous(), \
        dy.sum(0)
