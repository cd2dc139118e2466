"""Plain float64 reference of the training-side operators (numpy).

Test infrastructure, like the rest of this package: definitions written out,
no code shared with the library. Each function returns the result and a bound
on what fp32 arithmetic may add to it (before the final rounding to the
output's type): `k` fp32 roundings of 2^-24 on every term that is summed.
"""
from __future__ import annotations

import numpy as np

EPS32 = 2.0 ** -24          # half a step of fp32, relative


def sigmoid(a):
    t = np.exp(-np.abs(a))
    return np.where(a >= 0, 1.0 / (1.0 + t), t / (1.0 + t))


def _units(x, t_isolated):
    n, d, h, w, c = x.shape
    return x.reshape((n * d, h * w, c) if t_isolated else (n, d * h * w, c))


def group_norm_fwd(x, groups, gamma, beta, *, eps, silu, t_isolated, k=128):
    """(y, stats [units, groups, 2], bound of y)."""
    x5 = np.asarray(x, np.float64)
    xu = _units(x5, t_isolated)
    u, p, c = xu.shape
    xg = xu.reshape(u, p, groups, c // groups)
    mean = xg.mean(axis=(1, 3), keepdims=True)
    var = ((xg - mean) ** 2).mean(axis=(1, 3), keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    h = (xg - mean) * rstd
    g4 = np.asarray(gamma, np.float64).reshape(1, 1, groups, -1)
    b4 = np.asarray(beta, np.float64).reshape(1, 1, groups, -1)
    a = h * g4 + b4
    # the mean is off by k roundings of the mean distance from a thread's first
    # value (at most the group's widest one), and itself rounded to fp32; rstd
    # by k roundings of the squares' mean about that value
    spread = np.abs(xg - mean).max(axis=(1, 3), keepdims=True)
    dm = k * EPS32 * 2.0 * spread + 2 * EPS32 * np.abs(mean)
    dr = k * EPS32 * 4.0 * spread ** 2 * rstd ** 2 + 4 * EPS32
    tol = np.abs(g4) * (dm * rstd + np.abs(h) * (dr + 8 * EPS32)) + 4 * EPS32 * np.abs(b4)
    y = a
    if silu:
        y = a * sigmoid(a)
        tol = 1.1 * tol + 8 * EPS32 * np.abs(y)      # the slope is below 1.1
    stats = np.stack([mean.reshape(u, groups), rstd.reshape(u, groups)], axis=-1)
    return y.reshape(x5.shape), stats, tol.reshape(x5.shape)


def group_norm_bwd(dy, x, groups, gamma, beta, stats, *, silu, t_isolated, k=128):
    """((dx, dgamma, dbeta), bounds of the three), with stats as given."""
    x5 = np.asarray(x, np.float64)
    xu = _units(x5, t_isolated)
    u, p, c = xu.shape
    shape = (u, p, groups, c // groups)
    xg, dg = xu.reshape(shape), _units(np.asarray(dy, np.float64), t_isolated).reshape(shape)
    mean, rstd = (np.asarray(stats, np.float64)[..., i].reshape(u, 1, groups, 1) for i in (0, 1))
    g4 = np.asarray(gamma, np.float64).reshape(1, 1, groups, -1)
    b4 = np.asarray(beta, np.float64).reshape(1, 1, groups, -1)
    h = (xg - mean) * rstd
    a = h * g4 + b4
    slope = np.ones_like(a)
    if silu:
        s = sigmoid(a)
        slope = s + a * s * (1.0 - s)
    da = dg * slope
    N = p * (c // groups)
    db, dgm = da.sum(axis=1, keepdims=True), (da * h).sum(axis=1, keepdims=True)
    c1 = (g4 * db).sum(axis=3, keepdims=True) / N
    c2 = (g4 * dgm).sum(axis=3, keepdims=True) / N
    dx = rstd * (g4 * da - c1 - h * c2)
    # h: two roundings of x - mean and the product; a: two more; da through a
    # slope whose own slope is at most 1/2, and 8 roundings of the slope
    dh = 4 * EPS32 * np.abs(h)
    dda = np.zeros_like(h)
    if silu:
        dda = np.abs(dg) * (0.5 * (np.abs(g4) * dh + 4 * EPS32 * (np.abs(h * g4) + np.abs(b4)))
                            + 16 * EPS32)
    e1 = dda + k * EPS32 * np.abs(da)
    e2 = dda * np.abs(h) + np.abs(da) * dh + k * EPS32 * np.abs(da * h)
    t_db, t_dg = e1.sum(axis=1, keepdims=True), e2.sum(axis=1, keepdims=True)
    m1 = (np.abs(g4) * t_db).sum(axis=3, keepdims=True) / N + 2 * EPS32 * np.abs(c1)
    m2 = (np.abs(g4) * t_dg).sum(axis=3, keepdims=True) / N + 2 * EPS32 * np.abs(c2)
    t_dx = rstd * (np.abs(g4) * dda + m1 + np.abs(h) * m2 + dh * np.abs(c2)
                   + 6 * EPS32 * (np.abs(g4 * da) + np.abs(c1) + np.abs(h * c2)))
    out = (dx.reshape(x5.shape), dgm.sum(axis=0).reshape(c), db.sum(axis=0).reshape(c))
    tol = (t_dx.reshape(x5.shape), t_dg.sum(axis=0).reshape(c) + 2 * EPS32 * np.abs(out[1]),
           t_db.sum(axis=0).reshape(c) + 2 * EPS32 * np.abs(out[2]))
    return out, tol


def norm_silu_fwd(value, gamma):
    """The norm x sqrt(C) x gamma -> SiLU of `value`, without roundings."""
    v = np.asarray(value, np.float64)
    c = v.shape[-1]
    den = np.maximum(np.sqrt((v * v).sum(axis=-1, keepdims=True)), 1e-12)
    a = v / den * np.sqrt(c) * np.asarray(gamma, np.float64)
    return a * sigmoid(a)


def norm_silu_bwd(value, dy, gamma, dskip=None, k=128):
    """((dvalue, dgamma, dbias), bounds of the three)."""
    v = np.asarray(value, np.float64)
    c = v.shape[-1]
    v, dy2 = v.reshape(-1, c), np.asarray(dy, np.float64).reshape(-1, c)
    g = np.asarray(gamma, np.float64)
    norm = np.sqrt((v * v).sum(axis=1, keepdims=True))
    clamped = norm <= 1e-12
    s = np.sqrt(c) / np.where(clamped, 1e-12, norm)
    e = v * s
    a = e * g
    sg = sigmoid(a)
    slope = sg + a * sg * (1.0 - sg)
    da = dy2 * slope
    gr = da * g
    back = np.where(clamped, 0.0, (gr * e).sum(axis=1, keepdims=True) / c)
    dv = s * (gr - e * back)
    # |v|^2 sums c products: c roundings at most in the sum, half in the root
    ks = (c / 2 + 8) * EPS32
    dda = np.abs(dy2) * (0.5 * (ks + 4 * EPS32) * np.abs(a) + 16 * EPS32)
    e_gr = dda * np.abs(g) + 2 * EPS32 * np.abs(gr)
    e_back = (e_gr * np.abs(e) + (ks + (c + 4) * EPS32) * np.abs(gr * e)).sum(
        axis=1, keepdims=True) / c
    t_dv = s * (e_gr + np.abs(e) * e_back + (ks + 6 * EPS32)
                * (np.abs(gr) + 2 * np.abs(e * back)))
    if dskip is not None:
        sk = np.asarray(dskip, np.float64).reshape(-1, c)
        dv = dv + sk
        t_dv = t_dv + 2 * EPS32 * np.abs(sk)
    t_dg = (dda * np.abs(e) + (ks + k * EPS32) * np.abs(da * e)).sum(axis=0)
    t_db = (t_dv + k * EPS32 * np.abs(dv)).sum(axis=0)
    shape = np.asarray(value).shape
    return ((dv.reshape(shape), (da * e).sum(axis=0), dv.sum(axis=0)),
            (t_dv.reshape(shape), t_dg, t_db))
