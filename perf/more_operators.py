"""What is measured of training and serving beside the row operators of
``perf/operators.py``: activation checkpoints in 8 bits (MXINT8) with the
passes that write and read them, and low-rank adapters of many requests
beside a shared projection on 4-bit weights (MXFP4).

Each case is one pass through one operator on channels-last data: a row is
one token, or one pixel of an NHWC map, and its columns are the channels.
``run`` computes the plain form in 32 bits with elementary torch operations,
or, with ``own`` set, calls the package.

MXINT8: a block of 32 consecutive columns of a row shares a unit 2^(s - 127),
s the smallest whole number of at least 1 with max|x| <= 127 units; a value is
stored as x / unit rounded to the nearest whole number (ties to even).  Packed:
codes int8 [rows][Kp], Kp the columns rounded up to 32; scales
[rows][4 ceil(Kp / 128)], one byte s a block.

MXFP4: a block of 32 consecutive values along the contracted axis shares a
scale 2^(s - 127), s = clamp(floor(log2 max|x|) - 2 + 127, 0, 254); a value is
x / scale rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the
even code, larger values to 6) with its sign.  Packed: codes [rows][Kp / 2],
two a byte, the even column in the low half; scales [ceil(Kp / 128)][rows][4],
one byte s a block.

Adapters: row m of adapter g = ids[m] adds scale[g] * up[g]^T (down[g] x[m]) to
the projection's output, a row whose id is -1 nothing; down is [G][r][K], up
[G][r][N].
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token's activation kept and restored: latency
        dict(name="checkpoint, one token", op="checkpoint", rows=1, cols=4096, dtype="bf16", pad=0),
        # a layer's input over a training batch, of an odd width inside a wider buffer
        dict(name="checkpoint, 16384 ragged", op="checkpoint", rows=16384, cols=4101, dtype="bf16", pad=11),
        # a convolution's fp32 map, 16 x 56 x 56 x 64, normalised for a bf16 layer and kept for the gradient
        dict(name="norm, 56x56x64 map", op="norm", rows=50176, cols=64, dtype="fp32", out="bf16", pad=0),
        # the gradient over a long training batch from what the forward pass kept
        dict(name="norm bwd, 16384 tokens", op="norm_bwd", rows=16384, cols=4096, grad="bf16", pad=0),
        # the gradient of a pointwise layer on an odd number of pixels from its checkpointed input
        dict(name="linear bwd, 1000 pixels", op="linear_bwd", M=1000, N=512, K=130, dtype="fp32", grad="fp32"),
        # the gradient over a training batch
        dict(name="linear bwd, 8192 tokens", op="linear_bwd", M=8192, N=4096, K=4096, dtype="bf16", grad="bf16"),
        # one token of one request: latency
        dict(name="adapters, one token", op="adapters", M=1, N=4096, K=4096, r=16, G=8, order="mixed", dtype="bf16",
             out="bf16", save=False),
        # a serving batch: a token each of requests with different adapters, some with none
        dict(name="adapters, 61 requests", op="adapters", M=61, N=8000, K=4096, r=16, G=32, order="mixed",
             dtype="bf16", out="bf16", save=False),
        # ragged sequences of several users' fine-tuning, the input kept for the gradient
        dict(name="adapters, 2011 tokens kept", op="adapters", M=2011, N=4096, K=4096, r=64, G=5, order="runs",
             dtype="fp16", out="fp16", save=True),
        # long prompts
        dict(name="adapters, 8192 tokens", op="adapters", M=8192, N=8192, K=8192, r=16, G=4, order="runs",
             dtype="bf16", out="bf16", save=False),
        # the gradients of a small layer's adapters, odd sizes, from the input itself
        dict(name="adapters bwd, 777 pixels", op="adapters_bwd", M=777, N=1000, K=520, r=8, G=3, order="mixed",
             dtype="fp32", grad="fp32", kept=False),
        # a fine-tuning step of several adapters on one batch from the checkpointed input
        dict(name="adapters bwd, 8192 tokens", op="adapters_bwd", M=8192, N=4096, K=4096, r=16, G=4, order="runs",
             dtype="bf16", grad="bf16", kept=True),
    ]


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    def kind():
        return rng.choice(sorted(TYPES))

    op = rng.choice(["checkpoint", "norm", "norm_bwd", "linear_bwd", "adapters", "adapters", "adapters_bwd"])
    if op in ("checkpoint", "norm", "norm_bwd"):
        cols = size(16, 8192)
        c = dict(op=op, rows=size(1, min(65536, 2 ** 26 // cols)), cols=cols, pad=rng.choice([0, 0, rng.randrange(1, 64)]))
        if op == "norm":
            c.update(dtype=kind(), out=kind())
        elif op == "norm_bwd":
            c.update(grad=kind())
        else:
            c.update(dtype=kind())
        return c
    if op == "linear_bwd":
        return dict(op=op, M=size(16, 8192), N=size(16, 4096), K=size(16, 4096), dtype=kind(), grad=kind())
    r, most = size(1, 128), 8192 if op == "adapters" else 4096
    c = dict(op=op, M=size(1, 8192), N=size(16, most), K=size(16, most), r=r, G=size(1, max(1, 512 // r)),
             order=rng.choice(["runs", "mixed"]), dtype=kind())
    if op == "adapters":
        c.update(out=kind(), save=rng.random() < 0.5)
    else:
        c.update(grad=kind(), kept=rng.random() < 0.5)
    return c


# ---- both formats in plain torch -------------------------------------------

def _blocks(x):
    """fp32 [rows, blocks, 32], zeros past the last column."""
    k = x.shape[1]
    kp = -(-k // 32) * 32
    y = torch.zeros(x.shape[0], kp, device=x.device)
    y[:, :k] = x
    return y.view(x.shape[0], kp // 32, 32)


def _power(s):
    """2^(s - 127) in fp32 for whole s of 0 to 254."""
    return torch.where(s > 0, s << 23, torch.full_like(s, 1 << 22)).to(torch.int32).view(torch.float32)


def _whole_dwords(s):
    """A byte a block, [rows, blocks], filled up with zeros to whole dwords a row."""
    n, nb = s.shape
    scales = torch.zeros(n, -(-nb // 4) * 4, dtype=torch.uint8, device=s.device)
    scales[:, :nb] = s.to(torch.uint8)
    return scales


def _pack8(x):
    """codes and scales of fp32 rows in MXINT8."""
    b = _blocks(x)
    # the exponent field, one more where the mantissa is above 127 / 64: then 127 units of the field's own do not do
    s = ((b.abs().amax(-1).view(torch.int32) + 0x1ffff >> 23) - 6).clamp_min(1)
    return torch.round(b * _power(254 - s).unsqueeze(-1)).to(torch.int8).view(x.shape[0], -1), _whole_dwords(s)


def _values8(codes, scales, k):
    """fp32 [rows, K]"""
    n = codes.shape[0]
    c = codes.view(n, -1, 32).float()
    return (c * _power(scales[:, :c.shape[1]].int()).unsqueeze(-1)).view(n, -1)[:, :k]


def _scale_bytes4(b):
    return ((b.abs().amax(-1).view(torch.int32) >> 23) - 2).clamp_min(0)


def _rounded4(b, s):
    """The blocks over their scales, rounded to the grid."""
    v = b * _power(254 - s).unsqueeze(-1)
    a = v.abs()
    r = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return torch.copysign(r.clamp_max(6), v)


def _fake4(x):
    """fp32 [rows, K]: what the rows in MXFP4 stand for."""
    b = _blocks(x)
    s = _scale_bytes4(b)
    return (_rounded4(b, s) * _power(s).unsqueeze(-1)).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _pack4(w):
    """codes and scales of fp32 rows, as a program keeps its weights."""
    b = _blocks(w)
    s = _scale_bytes4(b)
    r = _rounded4(b, s)
    a = r.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(r).to(torch.uint8) << 3)).view(b.shape[0], -1, 2)
    scales = _whole_dwords(s).view(b.shape[0], -1, 4).permute(1, 0, 2).contiguous()
    return code[:, :, 0] | (code[:, :, 1] << 4), scales


def _values4(codes, scales, k):
    n = codes.shape[0]
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    q = torch.stack((codes & 15, codes >> 4), -1).to(torch.int32).reshape(n, -1, 32)
    s = scales.permute(1, 0, 2).reshape(n, -1)[:, :q.shape[1]].int()
    return (torch.cat((v, -v))[q] * _power(s).unsqueeze(-1)).reshape(n, -1)[:, :k]


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


def _ids(gen, case):
    """An adapter a row: requests' rows one after another, or any order; about one request in eight has none."""
    M, G = case["M"], case["G"]
    if case["order"] == "mixed":
        ids = torch.randint(0, G, (M,), generator=gen, device="cuda")
        none = torch.rand(M, generator=gen, device="cuda") < 0.125
        none[0] = False
    else:
        runs = 2 * G
        cuts = torch.sort(torch.randint(0, M, (runs - 1,), generator=gen, device="cuda")).values
        request = torch.searchsorted(cuts, torch.arange(M, device="cuda"), right=True)
        ids = torch.randint(0, G, (runs,), generator=gen, device="cuda")[request]
        none = (torch.rand(runs, generator=gen, device="cuda") < 0.125)[request]
        none &= none.logical_not().any()
    return torch.where(none, -1, ids).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op in ("checkpoint", "norm"):
        s["x"] = _rows(gen, case["rows"], case["cols"], case["dtype"], case["pad"])
    if op in ("norm", "norm_bwd"):
        s["gamma"] = 1 + 0.1 * torch.randn(case["cols"], generator=gen, device="cuda")
        s["beta"] = 0.1 * torch.randn(case["cols"], generator=gen, device="cuda")
    if op == "norm_bwd":
        s["dy"] = _grads(gen, case["rows"], case["cols"], case["grad"], case["pad"])
        n, _, s["rstd"] = _norm(_rows(gen, case["rows"], case["cols"], "fp32"))
        s["codes"], s["scales"] = _pack8(n)
    if op in ("linear_bwd", "adapters", "adapters_bwd"):
        M, N, K = case["M"], case["N"], case["K"]
        x = _rows(gen, M, K, case["dtype"])
        w = torch.randn(N, K, generator=gen, device="cuda") / math.sqrt(K)
    if op == "linear_bwd":
        s["w"] = w.to(TYPES[case["dtype"]])
        s["codes"], s["scales"] = _pack8(x.float())
        s["dy"] = _grads(gen, M, N, case["grad"])
    if op in ("adapters", "adapters_bwd"):
        G, r, t = case["G"], case["r"], TYPES[case["dtype"]]
        s["down"] = (torch.randn(G, r, K, generator=gen, device="cuda") / math.sqrt(K)).to(t)
        s["up"] = (0.5 * torch.randn(G, r, N, generator=gen, device="cuda") / math.sqrt(r)).to(t)
        s["scale"] = 0.5 + torch.rand(G, generator=gen, device="cuda")
        s["ids"] = _ids(gen, case)
    if op == "adapters":
        s["x"] = x
        s["wcodes"], s["wscales"] = _pack4(w)
        s["bias"] = 0.1 * torch.randn(N, generator=gen, device="cuda")
    if op == "adapters_bwd":
        s["wcodes"], s["wscales"] = _pack4(w.t())
        s["dy"] = _grads(gen, M, N, case["grad"])
        if case["kept"]:
            s["codes"], s["scales"] = _pack8(x.float())
        else:
            s["x"] = x
        s["h"] = _through(x.float(), s["down"], s["ids"])
    return s


# ---- one pass -------------------------------------------------------------

def _norm(x):
    x = x.float()
    mean = x.mean(-1)
    c = x - mean[:, None]
    rstd = torch.rsqrt(c.square().mean(-1) + EPS)
    return c * rstd[:, None], mean, rstd


def _through(x, m, ids):
    """[rows, r]: each row times its own adapter's [r, columns], 0 without one."""
    G, r, k = m.shape
    every = torch.matmul(x, m.float().reshape(G * r, k).t()).view(-1, G, r)
    mine = torch.gather(every, 1, ids.clamp_min(0).long()[:, None, None].expand(-1, 1, r))[:, 0]
    return torch.where(ids[:, None] >= 0, mine, 0.0)


def _spread(h, ids, G):
    """[rows, G r]: each row's values at its own adapter's place, zeros elsewhere."""
    at = torch.arange(G, device=h.device)[None, :, None] == ids[:, None, None]
    return torch.where(at, h[:, None, :], 0.0).reshape(h.shape[0], -1)


def _own_scale(scale, ids):
    return scale[ids.clamp_min(0).long()][:, None]


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    op = c["op"]
    if op == "checkpoint":
        x = state["x"]
        codes, scales = _pack8(x.float())
        return _values8(codes, scales, x.shape[1]).to(x.dtype)
    if op == "norm":
        n, _, rstd = _norm(state["x"])
        y = n * state["gamma"] + state["beta"]
        codes, scales = _pack8(n)
        return y.to(TYPES[c["out"]]), _values8(codes, scales, n.shape[1]).bfloat16(), rstd
    if op == "norm_bwd":
        dy = state["dy"].float()
        n = _values8(state["codes"], state["scales"], c["cols"])
        g = dy * state["gamma"]
        dx = state["rstd"][:, None] * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
        return dx.to(state["dy"].dtype), (dy * n).sum(0), dy.sum(0)
    if op == "linear_bwd":
        dy, w = state["dy"].float(), state["w"].float()
        x = _values8(state["codes"], state["scales"], c["K"])
        dx = torch.matmul(_fake4(dy), _fake4(w.t()).t())
        dw = torch.matmul(_fake4(dy.t()), _fake4(x.t()).t())
        return dx.to(state["w"].dtype), dw, dy.sum(0)
    ids, G, r = state["ids"], c["G"], c["r"]
    down, up = state["down"].float().view(G * r, -1), state["up"].float().view(G * r, -1)
    if op == "adapters":
        x = state["x"].float()
        h = _through(x, state["down"], ids)
        y = torch.matmul(_fake4(x), _values4(state["wcodes"], state["wscales"], c["K"]).t()) + state["bias"]
        y = (y + torch.matmul(_spread(h * _own_scale(state["scale"], ids), ids, G), up)).to(TYPES[c["out"]])
        if not c["save"]:
            return y
        codes, scales = _pack8(x)
        return y, _values8(codes, scales, c["K"]).bfloat16(), h
    dy = state["dy"].float()
    x = _values8(state["codes"], state["scales"], c["K"]) if c["kept"] else state["x"].float()
    s = _own_scale(state["scale"], ids)
    t = _through(dy, state["up"], ids) * s
    dx = torch.matmul(_fake4(dy), _values4(state["wcodes"], state["wscales"], c["N"]).t())
    ts = _spread(t, ids, G)
    ddown = torch.matmul(ts.t(), x).view(G, r, -1)
    dup = torch.matmul(_spread(state["h"] * s, ids, G).t(), dy).view(G, r, -1)
    return (dx + torch.matmul(ts, down)).to(state["dy"].dtype), ddown, dup


def _run_own(state):
    import convolution_implicit_gemm_fwd_amd as cim

    c = state["case"]
    op = c["op"]
    if op == "checkpoint":
        return cim.mxint8_dequantize_nhwc(cim.mxint8_quantize_nhwc(state["x"]), state["x"].dtype)
    if op == "norm":
        y, kept, rstd = cim.layer_norm_mxint8_nhwc(state["x"], state["gamma"], state["beta"], eps=EPS,
                                                   out_dtype=TYPES[c["out"]])
        return y, cim.mxint8_dequantize_nhwc(kept, torch.bfloat16), rstd
    if op == "norm_bwd":
        kept = cim.Mxint8Tensor(state["codes"], state["scales"], c["rows"], c["cols"])
        return cim.layer_norm_bwd_mxint8_nhwc(state["dy"], kept, state["gamma"], state["rstd"])
    if op == "linear_bwd":
        kept = cim.Mxint8Tensor(state["codes"], state["scales"], c["M"], c["K"])
        return cim.mxfp4_linear_bwd_nhwc(state["dy"], kept, state["w"])
    adapters = cim.Adapters(state["down"], state["up"], state["scale"])
    if op == "adapters":
        w = cim.Mxfp4Tensor(state["wcodes"], state["wscales"], c["N"], c["K"])
        out = cim.mxfp4_linear_adapters_nhwc(state["x"], w, state["bias"], adapters, state["ids"],
                                             out_dtype=TYPES[c["out"]], save=c["save"])
        return (out[0], cim.mxint8_dequantize_nhwc(out[1], torch.bfloat16), out[2]) if c["save"] else out
    wt = cim.Mxfp4Tensor(state["wcodes"], state["wscales"], c["K"], c["N"])
    x = cim.Mxint8Tensor(state["codes"], state["scales"], c["M"], c["K"]) if c["kept"] else state["x"]
    return cim.mxfp4_linear_adapters_bwd_nhwc(state["dy"], x, wt, adapters, state["ids"], state["h"])


# ---- what a pass cannot do without ---------------------------------------

def work(case):
    def b(t):
        return TYPES[t].itemsize

    def q8(rows, cols):
        return rows * -(-cols // 32) * 33

    def q4(rows, cols):
        return rows * -(-cols // 32) * 17

    op = case["op"]
    if op in ("checkpoint", "norm", "norm_bwd"):
        r, k = case["rows"], case["cols"]
        e = r * k
        if op == "checkpoint":
            return dict(bytes=2 * e * b(case["dtype"]) + 2 * q8(r, k), flops=4 * e)
        if op == "norm":      # (the kept values are restored, too)
            return dict(bytes=e * (b(case["dtype"]) + b(case["out"])) + 2 * q8(r, k) + 2 * e + 8 * k + 4 * r, flops=12 * e)
        return dict(bytes=2 * e * b(case["grad"]) + q8(r, k) + 12 * k + 4 * r, flops=14 * e)
    M, N, K = case["M"], case["N"], case["K"]
    if op == "linear_bwd":
        return dict(bytes=M * N * b(case["grad"]) + q8(M, K) + M * K * b(case["dtype"]) + N * K * (b(case["dtype"]) + 4)
                    + 4 * N, flops=4 * M * N * K)
    G, r, t = case["G"], case["r"], b(case["dtype"])
    ab = min(G, M) * r * (N + K)
    if op == "adapters":
        kept = (2 * q8(M, K) + 2 * M * K + 4 * M * r) if case["save"] else 0
        return dict(bytes=M * K * t + q4(N, K) + ab * t + M * N * b(case["out"]) + 4 * N + 8 * M + kept,
                    flops=2 * M * N * K + 2 * M * r * (N + K))
    x = q8(M, K) if case["kept"] else M * K * t
    return dict(bytes=M * N * b(case["grad"]) + x + q4(K, N) + ab * t + M * K * b(case["grad"]) + 4 * G * r * (N + K)
                + M * (8 + 4 * r), flops=2 * M * N * K + 4 * M * r * (N + K))


# ---- the definitions in 64 bits -------------------------------------------

def _exact_power(e):
    """2^e in fp64 for whole e, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _padded(x):
    return torch.nn.functional.pad(x, (0, -x.shape[1] % 32)).reshape(x.shape[0], -1, 32)


def _exact_fake8(x):
    """The smallest unit of which 127 reach the block's largest magnitude m 2^e, 1/2 <= m < 1, then whole units."""
    b = _padded(x)
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    unit = _exact_power((e - 7 + (m * 128 > 127)).clamp_min(-126))
    a = b / unit
    low = torch.floor(a)
    rest = a - low
    up = (rest > 0.5) | ((rest == 0.5) & (torch.remainder(low, 2) == 1))
    return ((low + up) * unit).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _exact_values8(codes, scales, k):
    return codes[:, :k].double() * _exact_power(scales.long().repeat_interleave(32, 1)[:, :k] - 127)


def _exact_fake4(x):
    """Along the last axis, by thresholds between neighbouring grid values."""
    b = _padded(x)
    _, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = torch.where((b == 0).all(-1, keepdim=True), torch.full_like(e, -200), e - 3).clamp(-127, 127)
    unit = _exact_power(e)
    a = b.abs() / unit
    q = 0.5 * ((a > 0.25).double() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) \
        + (a > 2.5).double() + (a >= 3.5).double() + 2 * (a > 5).double()
    return (torch.sign(b) * q * unit).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _exact_values4(codes, scales, k):
    q = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.long, device=codes.device)
    q[:, 0::2], q[:, 1::2] = codes.long() % 16, codes.long() // 16
    q = q[:, :k]
    e, m = (q % 8) // 2, (q % 2).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * _exact_power(e - 1))
    c = torch.arange(k, device=codes.device)
    return torch.where(q >= 8, -mag, mag) * _exact_power(scales.long()[c // 128, :, (c // 32) % 4].t() - 127)


def _exact_adapters(x, first, second, scale, ids):
    """(first_g x, scale_g second_g^T first_g x) a row, by adapter."""
    h = torch.zeros(x.shape[0], first.shape[1], dtype=torch.float64, device=x.device)
    out = torch.zeros(x.shape[0], second.shape[2], dtype=torch.float64, device=x.device)
    for g in range(first.shape[0]):
        mine = (ids == g).nonzero()[:, 0]
        h[mine] = x[mine] @ first[g].double().t().contiguous()
        out[mine] = scale[g].double() * (h[mine] @ second[g].double())
    return h, out


def _exact_sums(h, x, scale, ids):
    """scale_g * sum over the adapter's rows of h x^T, [G, r, columns]."""
    out = torch.zeros(scale.shape[0], h.shape[1], x.shape[1], dtype=torch.float64, device=x.device)
    for g in range(scale.shape[0]):
        mine = (ids == g).nonzero()[:, 0]
        out[g] = scale[g].double() * (h[mine].t().contiguous() @ x[mine])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "checkpoint":
        return _exact_fake8(s["x"].double())
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        n = (x - mean) / (var + EPS).sqrt()
        return n * s["gamma"].double() + s["beta"].double(), _exact_fake8(n), (var[:, 0] + EPS) ** -0.5
    if op == "norm_bwd":
        dy, n = s["dy"].double(), _exact_values8(s["codes"], s["scales"], case["cols"])
        h, k = dy * s["gamma"].double(), case["cols"]
        return s["rstd"].double()[:, None] / k * (k * h - h.sum(-1, keepdim=True) - n * (h * n).sum(-1, keepdim=True)), \
            (dy * n).sum(0), dy.sum(0)
    if op == "linear_bwd":
        dy, w = s["dy"].double(), s["w"].double()
        x = _exact_values8(s["codes"], s["scales"], case["K"])
        dyt, xt, wt = (t.t().contiguous() for t in (dy, x, w))
        return _exact_fake4(dy) @ _exact_fake4(wt).t().contiguous(), \
            _exact_fake4(dyt) @ _exact_fake4(xt).t().contiguous(), dy.sum(0)
    if op == "adapters":
        x = s["x"].double()
        w = _exact_values4(s["wcodes"], s["wscales"], case["K"])
        h, more = _exact_adapters(x, s["down"], s["up"], s["scale"], s["ids"])
        y = _exact_fake4(x) @ w.t().contiguous() + s["bias"].double() + more
        return (y, _exact_fake8(x), h) if case["save"] else y
    dy = s["dy"].double()
    x = _exact_values8(s["codes"], s["scales"], case["K"]) if case["kept"] else s["x"].double()
    w = _exact_values4(s["wcodes"], s["wscales"], case["N"])
    t, more = _exact_adapters(dy, s["up"], s["down"], s["scale"], s["ids"])
    return _exact_fake4(dy) @ w.t().contiguous() + more, _exact_sums(t, x, s["scale"], s["ids"]), \
        _exact_sums(s["h"].double(), dy, s["scale"], s["ids"])
