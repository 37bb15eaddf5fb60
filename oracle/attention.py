"""Reference oracle for the attention kernels (fp64, CPU).

TEST INFRASTRUCTURE ONLY: imported by the test suite and ``__graft_entry__``'s
smoke check, never by the product path.

Plain numpy in float64, written from the definitions in include/attention.h:
attention over packed sequences and its gradients, and the norm and rotation
of query and key heads and its gradients.  Every function also returns how
far an fp32 evaluation may be off, element by element, from a count of its
roundings (u = 2^-24): a sum of n products is off by at most (n + 1) u times
the sum of their magnitudes, in any order; exp2, log2, rsqrt, sine and cosine
are taken as good to 4 u.  Pinned by tests/test_oracle_attention.py.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def sequences(cu, tokens):
    """The [first, behind) rows of every sequence (None: one of all rows)."""
    if cu is None:
        return [(0, tokens)]
    c = np.clip(np.asarray(cu, dtype=np.int64), 0, tokens)
    return [(int(a), int(max(a, b))) for a, b in zip(c[:-1], c[1:])]


def visible(n, causal, window):
    i = np.arange(n)
    gap = i[:, None] - i[None, :]
    see = np.ones((n, n), dtype=bool)
    if causal:
        see &= gap >= 0
    if window:
        see &= np.abs(gap) < window
    return see


def _score_error(q, k, s, scale):
    """How far scale q.k may be off in fp32, scores going through exp2."""
    d = q.shape[1]
    return scale * (d + 4) * U * (np.abs(q) @ np.abs(k).T) + 8 * U * np.abs(s)


def attention(q, k, v, cu=None, causal=True, window=0, scale=None):
    """out [T, Hq, D], lse [Hq, T], and their bounds (out_err, lse_err)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    T, hq, d = q.shape
    group = hq // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out, out_err = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    lse, lse_err = np.full((hq, T), -np.inf), np.zeros((hq, T))
    for a, b in sequences(cu, T):
        n = b - a
        if n == 0:
            continue
        see = visible(n, causal, window)
        for h in range(hq):
            qs, ks, vs = q[a:b, h], k[a:b, h // group], v[a:b, h // group]
            s = np.where(see, scale * (qs @ ks.T), -np.inf)
            top = s.max(1, keepdims=True)
            e = np.exp(s - top)
            total = e.sum(1, keepdims=True)
            p = e / total
            ds = np.where(see, _score_error(qs, ks, np.where(see, s, 0.0), scale), 0.0).max(1, keepdims=True)
            # the reference that is subtracted from the scores is rounded too
            ds = ds + 8 * U * np.abs(top)
            out[a:b, h] = p @ vs
            out_err[a:b, h] = (2 * ds + (2 * n + 24) * U) * (p @ np.abs(vs)) + 1e-37
            lse[h, a:b] = (top + np.log(total))[:, 0]
            lse_err[h, a:b] = (ds + (n + 16) * U + 8 * U * np.abs(top) + 8 * U * np.abs(np.log(total)))[:, 0]
    return out, lse, out_err, lse_err


def attention_backward(dout, q, k, v, out, lse, cu=None, causal=True, window=0, scale=None):
    """(dq, dk, dv) and their bounds, from the given out and lse."""
    dout, q, k, v, out, lse = (np.asarray(x, dtype=np.float64) for x in (dout, q, k, v, out, lse))
    T, hq, d = q.shape
    group = hq // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    grads = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)]
    errs = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)]
    for a, b in sequences(cu, T):
        n = b - a
        if n == 0:
            continue
        see = visible(n, causal, window)
        rows = n * group
        for h in range(hq):
            hk = h // group
            qs, ks, vs, gs, os_ = q[a:b, h], k[a:b, hk], v[a:b, hk], dout[a:b, h], out[a:b, h]
            s = scale * (qs @ ks.T)
            l = lse[h, a:b][:, None]
            p = np.where(see, np.exp(np.where(see, s - l, 0.0)), 0.0)
            dp, delta = gs @ vs.T, (gs * os_).sum(1, keepdims=True)
            ds = p * (dp - delta)
            rel = np.where(see, _score_error(qs, ks, s, scale) + 8 * U * np.abs(l) + 8 * U, 0.0)
            e_dp = (d + 2) * U * (np.abs(gs) @ np.abs(vs).T)
            e_delta = (d + 2) * U * (np.abs(gs) * np.abs(os_)).sum(1, keepdims=True)
            e_ds = p * ((rel + 4 * U) * np.abs(dp - delta) + (1 + rel) * (e_dp + e_delta))
            grads[0][a:b, h] += scale * (ds @ ks)
            errs[0][a:b, h] += scale * ((e_ds + (n + 6) * U * np.abs(ds)) @ np.abs(ks))
            grads[1][a:b, hk] += scale * (ds.T @ qs)
            errs[1][a:b, hk] += scale * ((e_ds + (rows + 6) * U * np.abs(ds)).T @ np.abs(qs))
            grads[2][a:b, hk] += p.T @ gs
            errs[2][a:b, hk] += (p * (rel + (rows + 6) * U)).T @ np.abs(gs)
    return (*grads, *[e + 1e-37 for e in errs])


def _angles(positions, inv_freq):
    """positions * inv_freq in extended precision (64-bit mantissa)."""
    return np.asarray(positions).astype(np.longdouble)[:, None] * np.asarray(inv_freq).astype(np.longdouble)[None, :]


def _pairs(d, rotated, interleaved):
    """The first and second dimension of every rotated pair."""
    p = np.arange(rotated // 2)
    return (2 * p, 2 * p + 1) if interleaved else (p, p + rotated // 2)


def qk_norm_rope(x, weight, positions, inv_freq, eps=1e-6, interleaved=False):
    """The norm and rotation of x [T, H, D]: (y, its bound)."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    d = x.shape[2]
    r = 1.0 / np.sqrt((x * x).mean(2, keepdims=True) + eps)
    n = x * r * w
    # r: a sum of d squares, halved by the root; three products
    rel = ((d + 6) / 2 + 12) * U
    y, err = n.copy(), np.abs(n) * rel
    angle = _angles(positions, inv_freq)
    c, s = (f(angle).astype(np.float64)[:, None] for f in (np.cos, np.sin))
    a, b = _pairs(d, 2 * angle.shape[1], interleaved)
    na, nb = n[..., a], n[..., b]
    y[..., a], y[..., b] = na * c - nb * s, nb * c + na * s
    # sine and cosine 4 u and the correction by the angle's rest 2 u, the combination 3 u, and 3 u to spare
    err[..., a] = err[..., b] = (np.abs(na) + np.abs(nb)) * (rel + 12 * U)
    return y, err + 1e-37


def qk_norm_rope_backward(dy, x, weight, positions, inv_freq, eps=1e-6, interleaved=False):
    """(dx, dweight, dx's bound, dweight's bound)."""
    dy, x, w = (np.asarray(v, dtype=np.float64) for v in (dy, x, weight))
    T, H, d = x.shape
    angle = _angles(positions, inv_freq)
    c, s = (f(angle).astype(np.float64)[:, None] for f in (np.cos, np.sin))
    a, b = _pairs(d, 2 * angle.shape[1], interleaved)
    dn, e_dn = dy.copy(), np.zeros_like(dy)
    ga, gb = dy[..., a], dy[..., b]
    dn[..., a], dn[..., b] = ga * c + gb * s, gb * c - ga * s
    e_dn[..., a] = e_dn[..., b] = (np.abs(ga) + np.abs(gb)) * 12 * U
    r = 1.0 / np.sqrt((x * x).mean(2, keepdims=True) + eps)
    rel_r = ((d + 6) / 2 + 6) * U
    n, g = x * r, dn * w
    e_g = e_dn * np.abs(w) + 2 * U * np.abs(g)
    mean = (g * n).mean(2, keepdims=True)
    size = (np.abs(g) * np.abs(n)).mean(2, keepdims=True)
    e_mean = (e_g * np.abs(n)).mean(2, keepdims=True) + (d + 6) * U * size
    dx = r * (g - n * mean)
    e_dx = r * (e_g + np.abs(n) * e_mean + (np.abs(g) + np.abs(n) * size) * (3 * rel_r + 8 * U))
    dw = (dn * n).sum((0, 1))
    # fp32 over the heads of a token, 64 bits from there, one rounding
    e_dw = (e_dn * np.abs(n) + np.abs(dn * n) * (rel_r + (H + 6) * U)).sum((0, 1)) + 2 * U * np.abs(dw)
    return dx, dw, e_dx + 1e-37, e_dw + 1e-37


def compare(y, ref, bound):
    """The largest |y - ref| / bound, and how many values exceed their bound
    (values that are not finite have to be equal)."""
    y, ref = np.asarray(y, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    fine = np.isfinite(ref)
    same = np.array_equal(y[~fine], ref[~fine], equal_nan=True)
    far = np.abs(y[fine] - ref[fine])
    # a bound of zero (rows of no sequence) asks for the exact value
    ratio = np.where(far == 0, 0.0, far / np.maximum(np.broadcast_to(bound, ref.shape)[fine], 1e-300))
    ratio = np.where(np.isnan(ratio), np.inf, ratio)
    return {"max_ratio": float(ratio.max()) if ratio.size else 0.0,
            "fails": int((ratio > 1).sum()) + (0 if same else 1), "n": int(ref.size)}
