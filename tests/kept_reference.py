"""Definitions in 64 bits (numpy, CPU) of what is kept in 8 bits and of the
low-rank adapters, with the tolerances that follow, beside row_reference.py.

A product of matrix instructions takes values of more than 8 bits as bf16 terms
(fp16 2, fp32 3): what it leaves out is below 2 u of a product, and a sum over n
columns is a chain of at most 6 n / 32 additions, the 32 inside an instruction
and the tree over waves and parts.
"""
import numpy as np

import row_reference as ref
from row_reference import HALF, TINY, U


def quantize(x):
    """(codes int8 [rows, kp], scales uint8 [rows, 4 quads], values [rows, cols], bad blocks [rows, blocks])."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = x
    b = b.reshape(rows, nb, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0, b)
    m, e = np.frexp(np.abs(b).max(-1))      # top = m 2^e with m in [1/2, 1), 0 for 0
    s = np.where(m == 0, 1, np.maximum(e - 7 + (m * 128 > 127) + 127, 1))
    unit = np.ldexp(1.0, s - 127)[..., None]
    codes = np.rint(b / unit)               # (to even)
    assert np.abs(codes).max(initial=0) <= 127
    val = np.where(bad[..., None], np.nan, codes * unit).reshape(rows, -1)[:, :cols]
    scales = np.zeros((rows, -(-nb // 4) * 4), np.uint8)
    scales[:, :nb] = np.where(bad, 255, s)
    return codes.astype(np.int8).reshape(rows, -1), scales, val, bad


def values(q):
    """What an Mxint8Tensor's rows stand for."""
    s = q.scales.cpu().numpy().astype(np.int64).repeat(32, 1)[:, :q.cols]
    return q.codes.cpu().numpy()[:, :q.cols].astype(np.float64) * np.ldexp(1.0, s - 127)


def norm(x, eps):
    """n, rstd and their tolerances (row_reference.layer_norm derives them)."""
    mean = x.mean(-1, keepdims=True)
    var = ((x - mean) ** 2).mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(var + eps)
    n = (x - mean) * rstd
    d = ref.chain(x.shape[-1])
    dm = (d + 1) * U * np.abs(x).mean(-1, keepdims=True)
    dr = ((d + 6) * U + np.minimum(dm ** 2 / (var + eps), 1)) / 2 + 3 * U
    return n, rstd[:, 0], rstd * dm + np.abs(n) * (dr + 3 * U), (rstd * dr)[:, 0]


def check_kept(q, n, dn, what):
    """The rows kept of n, known to dn: the unit is the smallest that reaches the block's largest magnitude, and a
    value is off by at most half of it."""
    rows, cols = n.shape
    nb = -(-cols // 32)
    s = q.scales.cpu().numpy().astype(np.int64)
    assert not s[:, nb:].any(), "%s: bytes past the last block" % what
    u = np.ldexp(1.0, s[:, :nb] - 127)
    def blocks(v):
        b = np.zeros((rows, nb * 32))
        b[:, :cols] = v
        return b.reshape(rows, nb, 32)
    top, slack = np.abs(blocks(n)).max(-1), blocks(dn).max(-1)
    assert (127 * u >= top - slack).all(), "%s: a unit is too small" % what
    assert ((s[:, :nb] == 1) | (127 * u / 2 < top + slack)).all(), "%s: a unit is too large" % what
    off = np.abs(values(q) - n) - dn
    half = (u / 2).repeat(32, 1)[:, :cols]
    assert (off <= half * (1 + 1e-9)).all(), "%s: %d values off by more than half a unit" % (what, (off > half).sum())
    codes = q.codes.cpu().numpy()
    assert not codes[:, cols:].any(), "%s: codes past the last column" % what


def norm_bwd(dy, n, gamma, rstd, out):
    """dx, dgamma, dbeta and their tolerances; n and rstd are inputs."""
    h = dy * (1 if gamma is None else gamma)
    m1, m2 = h.mean(-1, keepdims=True), (h * n).mean(-1, keepdims=True)
    dx = rstd[:, None] * (h - m1 - n * m2)
    d = ref.chain(dy.shape[-1])
    a1, a2 = np.abs(h).mean(-1, keepdims=True), np.abs(h * n).mean(-1, keepdims=True)
    err = U * (np.abs(h) * 5 + (d + 6) * a1 + np.abs(n) * (d + 12) * a2 + 4 * (np.abs(m1) + np.abs(n * m2)))
    rows = dy.shape[0]
    k = (rows + 600 + 6) * U      # a thread's rows, then up to 512 parts
    return dx, (dy * n).sum(0), dy.sum(0), rstd[:, None] * err + HALF[out] * np.abs(dx) + TINY[out], \
        k * np.abs(dy * n).sum(0) + 1e-40, k * np.abs(dy).sum(0) + 1e-40


def chain(n):
    return 6 * n / 32 + 64


def own(ids, G):
    return [(g, np.nonzero(ids == g)[0]) for g in range(G)]


def through(x, first, ids):
    """Each row times its own adapter's matrix, and the tolerance."""
    h = np.zeros((x.shape[0], first.shape[1]))
    dh = np.zeros_like(h)
    for g, m in own(ids, first.shape[0]):
        h[m] = x[m] @ first[g].T
        dh[m] = (chain(x.shape[1]) + 4) * U * (np.abs(x[m]) @ np.abs(first[g]).T)
    return h, dh


def beside(base, dbase, sbase, x, first, second, scale, ids, out):
    """The product with the adapters' part, (y, tolerance, h, its tolerance); base: the product, dbase its tolerance in
    fp32 and sbase its terms' magnitudes."""
    h, dh = through(x, first, ids)
    y, tol = base.copy(), dbase.copy()
    for g, m in own(ids, first.shape[0]):
        s = scale[g]
        part = np.abs(s) * (np.abs(h[m]) @ np.abs(second[g]))
        y[m] += s * (h[m] @ second[g])
        tol[m] += np.abs(s) * (dh[m] @ np.abs(second[g])) + (chain(second.shape[1]) + chain(x.shape[1])) * U * part
    return y, tol + 8 * U * sbase + HALF[out] * np.abs(y) + TINY[out], h, dh


def grads(u, du, v, scale, ids):
    """[G, r, columns] sums over each adapter's rows of u v^T times its scale, and the tolerance."""
    G = len(scale)
    o = np.zeros((G, u.shape[1], v.shape[1]))
    d = np.zeros_like(o)
    for g, m in own(ids, G):
        s = scale[g]
        o[g] = s * (u[m].T @ v[m])
        d[g] = np.abs(s) * (du[m].T @ np.abs(v[m]) + (chain(len(m)) + 64 + 6) * U * (np.abs(u[m]).T @ np.abs(v[m]))) + 1e-40
    return o, d
