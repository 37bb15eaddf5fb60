"""Reference oracle for the norms around a block (fp64, CPU).

TEST INFRASTRUCTURE ONLY: imported by the test suite and ``__graft_entry__``'s
smoke check, never by the product path.

Plain numpy in float64, written from the definitions in include/block_norm.h.
Every function also returns how far an fp32 evaluation may be off, element by
element, from a count of its roundings (u = 2^-24).  A row's sum is a tree: a
value passes at most 16 additions in its lane, 6 across the lanes and 8 across
waves, so with its product it is off by at most 32 u of the sum of magnitudes;
a sum over rows passes at most 68 in fp32 (64 rows of a lane, 4 lanes) and is
taken in 64 bits from there; rsqrt is good to 2 u.  Pinned by
tests/test_oracle_block_norm.py.
"""
from __future__ import annotations

import numpy as np

from oracle.attention import compare, sequences  # noqa: F401

U = 2.0 ** -24
ROW, ROWS = 32 * U, 70 * U


def _f64(*arrays):
    return [None if a is None else np.asarray(a, dtype=np.float64) for a in arrays]


def _root(x, eps):
    """The reciprocal root mean square of every row, and how far it may be off relative to itself: half of the
    mean's error (the sum, 1 / width, eps, the product and the addition), and the function's."""
    return 1.0 / np.sqrt((x * x).mean(1, keepdims=True) + eps), ROW / 2 + 4 * U


def _gate_rows(gate, cu, T):
    """Each row's gate and its sequence, and which rows belong to one."""
    seq, used = np.zeros(T, dtype=np.int64), np.zeros(T, dtype=bool)
    for b, (first, behind) in enumerate(sequences(cu, T)):
        seq[first:behind], used[first:behind] = b, True
    if gate is None:
        return 1.0, seq, used
    if gate.ndim == 1:
        return gate[None], seq, used
    rows = np.zeros((T, gate.shape[1]))
    rows[used] = gate[seq[used]]
    return rows, seq, used


def block_norm(x, y=None, pre_weight=None, post_weight=None, gate=None, residual_scale=1.0, block_scale=1.0, cu=None,
               eps=1e-6):
    """(x_out, h, their bounds); h is None without pre_weight, x_out is x without y.  Rows of no sequence are zero."""
    x, y, pre, post, gate = _f64(x, y, pre_weight, post_weight, gate)
    g, _, used = _gate_rows(gate, cu, x.shape[0])
    used = used[:, None]
    x = np.where(used, x, 0.0)
    if y is None:
        out, err = x, np.zeros_like(x)
    else:
        n, rel = np.where(used, y, 0.0), 0.0
        if post is not None:
            r, rel = _root(n, eps)
            n, rel = n * r * post, rel + 2 * U
        term = block_scale * g * n
        out = residual_scale * x + term
        # the scales are rounded, and each side's products and the addition
        err = np.abs(residual_scale * x) * 3 * U + np.abs(term) * (rel + 4 * U)
    if pre is None:
        return out, None, err + 1e-37, None
    r, rel = _root(out, eps)
    h = out * r * pre
    # what x_out is off by: its own values, and the mean of squares through the root
    shift = (np.abs(out) * err).mean(1, keepdims=True) * r * r
    e_h = np.abs(r * pre) * err + np.abs(h) * (shift + rel + 3 * U)
    live = used & np.ones_like(out, dtype=bool)
    return (np.where(used, out, 0.0), np.where(live, h, 0.0), np.where(used, err, 0.0) + 1e-37 * live,
            np.where(live, e_h + 1e-37, 0.0))


def _norm_backward(g, e_g, x, r, rel):
    """The gradient of x r from g, and its bound."""
    mean = (g * x).mean(1, keepdims=True) * r * r
    size = (np.abs(g) * np.abs(x)).mean(1, keepdims=True) * r * r
    e_mean = (e_g * np.abs(x)).mean(1, keepdims=True) * r * r + size * (ROW + 2 * rel + 4 * U)
    dx = r * (g - x * mean)
    return dx, r * (e_g + np.abs(x) * e_mean + (np.abs(g) + np.abs(x) * size) * (rel + 4 * U))


def block_norm_backward(dx_out, dh, x_out, y=None, pre_weight=None, post_weight=None, gate=None, residual_scale=1.0,
                        block_scale=1.0, cu=None, eps=1e-6):
    """{name: (gradient, bound)} of dx, dy, dpre_weight, dpost_weight, dgate, those that there are."""
    dx_out, dh, x, y, pre, post, gate = _f64(dx_out, dh, x_out, y, pre_weight, post_weight, gate)
    T = x.shape[0]
    g, seq, used = _gate_rows(gate, cu, T)
    used = used[:, None]
    clean = lambda a: np.where(used, a, 0.0)  # noqa: E731
    res = {}
    dt = np.zeros_like(x) if dx_out is None else clean(dx_out)
    e_dt = np.zeros_like(dt)
    if pre is not None:
        x, dh = clean(x), clean(dh)
        r, rel = _root(x, eps)
        through, e = _norm_backward(dh * pre, np.abs(dh * pre) * U, x, r, rel)
        e_dt = e + (np.abs(dt) + np.abs(through)) * 2 * U
        dt = dt + through
        dw = dh * x * r
        res["dpre_weight"] = dw.sum(0), (np.abs(dw) * (ROWS + rel + 2 * U)).sum(0) + U * np.abs(dw.sum(0))
    res["dx"] = clean(residual_scale * dt), clean(np.abs(residual_scale) * (e_dt + 2 * U * np.abs(dt)) + 1e-37)
    if y is None:
        return res
    y = clean(y)
    u, e_u = block_scale * dt, np.abs(block_scale) * (e_dt + 2 * U * np.abs(dt))
    r, rel = _root(y, eps) if post is not None else (1.0, 0.0)
    n = y * r
    dn, e_dn = u * g, np.abs(g) * e_u + np.abs(u * g) * U
    if gate is not None:
        full = n if post is None else n * post
        dg = u * full
        e = e_u * np.abs(full) + np.abs(dg) * (ROWS + rel + 4 * U)
        if gate.ndim == 1:
            res["dgate"] = dg.sum(0), e.sum(0) + U * np.abs(dg.sum(0))
        else:
            total, bound = np.zeros(gate.shape), np.zeros(gate.shape)
            rows = np.flatnonzero(used[:, 0])
            np.add.at(total, seq[rows], dg[rows])
            np.add.at(bound, seq[rows], e[rows])
            res["dgate"] = total, bound + U * np.abs(total)
    if post is None:
        res["dy"] = clean(dn), clean(e_dn + 1e-37)
    else:
        dw = dn * n
        res["dpost_weight"] = dw.sum(0), ((e_dn * np.abs(n)) + np.abs(dw) * (ROWS + rel + 2 * U)).sum(0) \
            + U * np.abs(dw.sum(0))
        dy, e = _norm_backward(dn * post, e_dn * np.abs(post) + np.abs(dn * post) * U, y, r, rel)
        res["dy"] = clean(dy), clean(e + 1e-37)
    return {k: (v, b + 1e-37) if k.endswith(("weight", "gate")) else (v, b) for k, (v, b) in res.items()}
