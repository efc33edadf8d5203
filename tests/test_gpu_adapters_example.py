"""examples/adapters.py on the GPU: a fine-tuning step's outputs and every gradient against the chain rule in 64 bits on
the values that the step itself kept, the served requests, and that it runs."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import convolution_implicit_gemm_fwd_amd as cim
import kept_reference as kept
import row_reference as ref
from gpu_harness import need_gpu
from row_reference import HALF, U, f64

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapters.py")
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ex():
    need_gpu()
    spec = importlib.util.spec_from_file_location("adapters_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def decoded(q):
    return f64(cim.mxfp4_dequantize_nhwc(q, FP32))


@pytest.mark.parametrize("rows", [3, 61, 300])
def test_step(ex, rows):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    base, p = ex.Base(gen), ex.users(gen)
    x = torch.randn(rows, ex.K, generator=gen, device="cuda").bfloat16()
    ids = torch.randint(-1, ex.USERS, (rows,), generator=gen, device="cuda").int()
    dy = torch.randn(rows, ex.N, generator=gen, device="cuda").bfloat16()
    y, (kept_n, rstd, kept_x, h) = ex.forward(base, p, x, ids)
    g = ex.backward(base, p, ids, (kept_n, rstd, kept_x, h), dy)
    who = f64(ids).astype(np.int64)
    down, up, scale = (f64(t) for t in ex.adapters(p))

    # the norm's output n (bf16) and what is kept of it and of its input
    want, _, r, tol, _, dr = ref.layer_norm(f64(x), f64(p["gamma"]), f64(p["beta"]), ex.EPS, BF16)
    ref.check(rstd, r, dr, "rstd")
    nh, _, dnh, _ = kept.norm(f64(x), ex.EPS)
    kept.check_kept(kept_n, nh, dnh, "kept normalised rows")
    n8 = kept.values(kept_x)
    unit = np.ldexp(1.0, kept_x.scales.cpu().numpy().astype(np.int64) - 127).repeat(32, 1)[:, :ex.K]
    assert (np.abs(n8 - want) <= tol + unit / 2 * (1 + 1e-9)).all()
    n = ex.cim.layer_norm_nhwc(x, p["gamma"], p["beta"], ex.EPS)      # (the same bf16 values but for rounding's ties)
    hn, dh = kept.through(f64(n), down, who)
    # h comes from the norm's output, of which another call may round a value the other way
    ref.check(h, hn, dh + 2 * kept.through(HALF[BF16] * np.abs(f64(n)), np.abs(down), who)[0] + 1e-40, "h")

    # gradients from what was kept
    a = ref.mx_quantize(f64(dy))[2]
    wt = decoded(base.wt)
    mags = np.abs(a) @ np.abs(wt).T
    dn, ddn, t, dt = kept.beside(a @ wt.T, (ex.N / 32 + 40) * U * mags, mags, f64(dy), up, down, scale, who, BF16)
    ref.check(g["down"], *kept.grads(t, dt, n8, scale, who), "ddown")
    ref.check(g["up"], *kept.grads(f64(h), 0 * f64(h), f64(dy), scale, who), "dup")
    nn = kept.values(kept_n)
    # gamma's and beta's gradients pass dn's rounding and error on
    _, dg, db, _, eg, eb = kept.norm_bwd(dn, nn, f64(p["gamma"]), f64(rstd), FP32)
    ref.check(g["gamma"], dg, 2 * eg + (ddn * np.abs(nn)).sum(0), "dgamma")
    ref.check(g["beta"], db, 2 * eb + ddn.sum(0), "dbeta")


@pytest.mark.parametrize("rows", [1, 4, 90, 700])
def test_served_rows(ex, rows):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    base, p = ex.Base(gen), ex.users(gen)
    x = torch.randn(rows, ex.K, generator=gen, device="cuda").bfloat16()
    ids = torch.randint(-1, ex.USERS, (rows,), generator=gen, device="cuda").int()
    got = ex.Served(base, p)(x, ids)
    n = f64(ex.cim.layer_norm_nhwc(x, p["gamma"], p["beta"], ex.EPS))      # (the same call, so the same values)
    a, w, b = ref.mx_quantize(n)[2], decoded(base.w), f64(base.bias)
    mags = np.abs(a) @ np.abs(w).T + np.abs(b)
    down, up, scale = (f64(t) for t in ex.adapters(p))
    y, tol, _, _ = kept.beside(a @ w.T + b, (ex.K / 32 + 40) * U * mags, mags, n, down, up, scale, f64(ids).astype(np.int64), BF16)
    ref.check(got, y, tol, "served rows")


def test_runs():
    r = subprocess.run([sys.executable, PATH, "12"], capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "step   11" in r.stdout and "served requests" in r.stdout
