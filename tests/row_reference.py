"""The row operators' definitions in 64 bits (numpy, CPU) and the tolerances
that follow from them, for the GPU tests.

u = 2^-24 is half a step of fp32; HALF[dtype] half a step of an output type.
A sum of n fp32 terms whose chain of additions is d long is off by at most
d u times the sum of the terms' magnitudes.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def chain(cols):
    """Additions on the longest path of a row's sum: at most one thread's
    share of the row (a 256-thread workgroup at least every 8 columns), then
    the tree over lanes and waves."""
    return -(-cols // 256) + 8 + 16


def layer_norm(x, gamma, beta, eps, out):
    """y, mean, rstd and their tolerances."""
    mean = x.mean(-1, keepdims=True)
    var = ((x - mean) ** 2).mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(var + eps)
    n = (x - mean) * rstd
    g = np.ones(x.shape[-1]) if gamma is None else gamma
    b = np.zeros(x.shape[-1]) if beta is None else beta
    y = n * g + b
    d = chain(x.shape[-1])
    dm = (d + 1) * U * np.abs(x).mean(-1, keepdims=True)          # the mean: its sum, its division
    # the variance: the squares' sum and rounding, the mean's error (it adds dm^2
    # and the differences' own rounding, 2u each); rstd takes half of it
    dv = (d + 6) * U + np.minimum(dm ** 2 / (var + eps), 1)
    dr = dv / 2 + 3 * U
    # the difference's rounding is u |x - mean| + the mean's error
    dn = rstd * dm + np.abs(n) * (dr + 3 * U)
    dy = np.abs(g) * dn + 3 * U * (np.abs(y) + np.abs(b)) + HALF[out] * np.abs(y) + TINY[out]
    return y, mean[..., 0], rstd[..., 0], dy, dm[..., 0] + TINY[torch.float32], (rstd * dr)[..., 0]


def layer_norm_bwd(dy, x, gamma, mean, rstd, out, parts_chain):
    """dx, dgamma, dbeta and their tolerances; mean and rstd are inputs."""
    m, r = mean[:, None], rstd[:, None]
    n = (x - m) * r
    h = dy * (np.ones(x.shape[-1]) if gamma is None else gamma)
    m1, m2 = h.mean(-1, keepdims=True), (h * n).mean(-1, keepdims=True)
    dx = r * (h - m1 - n * m2)
    d = chain(x.shape[-1])
    a1, a2 = np.abs(h).mean(-1, keepdims=True), np.abs(h * n).mean(-1, keepdims=True)
    # n is off by 2u, h by u, a product by u; three more roundings at the end
    err = U * (np.abs(h) * 5 + (d + 6) * a1 + np.abs(n) * (d + 12) * a2 + 4 * (np.abs(m1) + np.abs(n * m2)))
    ddx = r * err + HALF[out] * np.abs(dx) + TINY[out]
    rows = x.shape[0]
    k = (parts_chain + 6) * U
    return dx, (dy * n).sum(0), dy.sum(0), ddx, k * np.abs(dy * n).sum(0) + 1e-40, k * np.abs(dy).sum(0) + 1e-40


def mx_quantize(x):
    """(codes uint8 [rows, kp/2], scales uint8 [quads, rows, 4], values [rows, cols])."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = x
    b = b.reshape(rows, nb, 32)
    bad = ~np.isfinite(b).all(-1)
    top = np.where(bad, 1, np.abs(np.where(np.isfinite(b), b, 0)).max(-1))
    # frexp gives top = m 2^e with m in [1/2, 1)
    s = np.where(top > 0, np.clip(np.frexp(np.where(top > 0, top, 1))[1] - 1 - 2 + 127, 0, 254), 0)
    v = np.where(bad[..., None], 0, b) / np.ldexp(1.0, s - 127)[..., None]
    a = np.abs(v)
    # the nearest grid value; a tie goes to the even code
    i = np.searchsorted(GRID, a, side="right") - 1
    j = np.minimum(i + 1, 7)
    lo, hi = a - GRID[i], GRID[j] - a
    code = np.where((hi < lo) | ((hi == lo) & (i % 2 == 1)), j, i)
    code = np.where(a >= 6, 7, code)
    neg = np.signbit(v)
    val = np.where(neg, -1, 1) * GRID[code] * np.ldexp(1.0, s - 127)[..., None]
    val = np.where(bad[..., None], np.nan, val).reshape(rows, -1)[:, :cols]
    code = (code + 8 * neg).astype(np.uint8).reshape(rows, -1)
    nq = -(-nb // 4)
    scales = np.zeros((rows, nq * 4), np.uint8)
    scales[:, :nb] = np.where(bad, 255, s)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales.reshape(rows, nq, 4).transpose(1, 0, 2).copy(), val, bad


def product(a, b, bias, out):
    """a b^T + bias and its tolerance: products of grid values are exact in
    fp32, a chain adds at most one product of 32 columns at a time, and the
    32 inside the matrix instruction."""
    y = a @ b.T + (0 if bias is None else bias)
    s = np.abs(a) @ np.abs(b).T + (0 if bias is None else np.abs(bias))
    d = a.shape[1] / 32 + 32 + 8
    return y, d * U * s + HALF[out] * np.abs(y) + TINY[out]


def check(got, want, tol, what):
    got = f64(got)
    assert got.shape == want.shape, "%s: shape %s, not %s" % (what, got.shape, want.shape)
    assert np.isfinite(got).all(), "%s: %d values not finite" % (what, (~np.isfinite(got)).sum())
    over = np.abs(got - want) > tol
    if over.any():
        k = np.unravel_index(np.argmax(np.where(over, np.abs(got - want) / tol, 0)), got.shape)
        raise AssertionError("%s: %d of %d outside the tolerance, worst at %s: %r for %r, tolerance %.3g"
                             % (what, over.sum(), over.size, k, got[k], want[k], np.broadcast_to(tol, got.shape)[k]))
