"""Pins of the block norm oracle (CPU): torch's float64 autograd, central
differences, closed forms, rows of no sequence, and planted mistakes that the
bounds have to catch."""
import numpy as np
import pytest

from oracle import block_norm as OB


def case(seed, T=11, W=7, post=True, gate="sequence", cu=(1, 4, 4, 9), a=0.9, b=0.4, pre=True):
    r = np.random.default_rng(seed)
    n = lambda *s: r.standard_normal(s)  # noqa: E731
    kw = dict(pre_weight=n(W) if pre else None, post_weight=n(W) if post else None, residual_scale=a, block_scale=b,
              cu=None if cu is None else np.array(cu), eps=1e-5,
              gate={"none": None, "shared": n(W), "sequence": n(len(cu) - 1 if cu else 1, W)}[gate])
    return n(T, W), n(T, W), n(T, W), n(T, W), kw


def torch_forward(x, y, kw):
    import torch
    norm = lambda v, w: v / torch.sqrt((v * v).mean(1, keepdim=True) + kw["eps"]) * w  # noqa: E731
    T = x.shape[0]
    out, h = torch.zeros_like(x), torch.zeros_like(x)
    for b, (s0, s1) in enumerate(OB.sequences(kw["cu"], T)):
        n = y[s0:s1]
        if kw["post_weight"] is not None:
            n = norm(n, kw["post_weight"])
        if kw["gate"] is not None:
            n = n * (kw["gate"] if kw["gate"].dim() == 1 else kw["gate"][b])
        o = kw["residual_scale"] * x[s0:s1] + kw["block_scale"] * n
        out = torch.cat((out[:s0], o, out[s1:]))
        if kw["pre_weight"] is not None:
            h = torch.cat((h[:s0], norm(o, kw["pre_weight"]), h[s1:]))
    return out, h


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("gate,cu", [("none", None), ("shared", None), ("shared", (0, 5, 9)), ("sequence", (1, 4, 4, 9)),
                                     ("sequence", (0, 11))])
def test_against_autograd(post, pre, gate, cu):
    import torch
    x, y, gx, gh, kw = case(3, post=post, gate=gate, cu=cu, pre=pre)
    t = {n: torch.tensor(a, requires_grad=True) for n, a in
         {"x": x, "y": y, **{k: kw[k] for k in ("pre_weight", "post_weight", "gate")}}.items() if a is not None}
    tk = dict(kw, **{k: t.get(k) for k in ("pre_weight", "post_weight", "gate")})
    out, h = torch_forward(t["x"], t["y"], tk)
    ro, rh, _, _ = OB.block_norm(x, y, **kw)
    assert np.allclose(ro, out.detach().numpy(), rtol=1e-13, atol=1e-13)
    loss = (out * torch.tensor(gx)).sum()
    if pre:
        assert np.allclose(rh, h.detach().numpy(), rtol=1e-13, atol=1e-13)
        loss = loss + (h * torch.tensor(gh)).sum()
    else:
        assert rh is None
    loss.backward()
    got = OB.block_norm_backward(gx, gh if pre else None, ro, y, **kw)
    names = {"dx": "x", "dy": "y", "dpre_weight": "pre_weight", "dpost_weight": "post_weight", "dgate": "gate"}
    assert set(got) == {k for k, v in names.items() if v in t}
    for k, (g, bound) in got.items():
        assert np.allclose(g, t[names[k]].grad.numpy(), rtol=1e-11, atol=1e-12), k
        assert g.shape == bound.shape and (bound >= 0).all()


def test_against_differences():
    x, y, gx, gh, kw = case(5)
    loss = lambda x, y, kw: sum((r * g).sum() for r, g in zip(OB.block_norm(x, y, **kw)[:2], (gx, gh)))  # noqa: E731
    got = OB.block_norm_backward(gx, gh, OB.block_norm(x, y, **kw)[0], y, **kw)
    r = np.random.default_rng(0)
    for name, key in (("dx", "x"), ("dy", "y"), ("dpre_weight", "pre_weight"), ("dpost_weight", "post_weight"),
                      ("dgate", "gate")):
        base = {"x": x, "y": y}.get(key, kw.get(key))
        step = r.standard_normal(base.shape)
        def at(e):
            moved = base + e * step
            if key in ("x", "y"):
                return loss(moved if key == "x" else x, moved if key == "y" else y, kw)
            return loss(x, y, dict(kw, **{key: moved}))
        slope = (at(1e-5) - at(-1e-5)) / 2e-5
        assert abs(slope - (got[name][0] * step).sum()) < 1e-7 * max(1.0, abs(slope)), name


def test_closed_forms():
    """A constant row has norm 1 (eps 0); without y the norm alone; the gradient of a norm is orthogonal to its row."""
    x = np.full((3, 5), -4.0)
    out, h, e, eh = OB.block_norm(x, pre_weight=np.arange(5.0), eps=0.0)
    assert np.array_equal(out, x) and np.allclose(h, -np.arange(5.0)[None])
    r = np.random.default_rng(1)
    v, g = r.standard_normal((4, 6)), r.standard_normal((4, 6))
    dx = OB.block_norm_backward(None, g, v, pre_weight=np.ones(6), eps=0.0)["dx"][0]
    assert np.abs((dx * v).sum(1)).max() < 1e-12


def test_rows_of_no_sequence():
    x, y, gx, gh, kw = case(7)
    x[[0, 9, 10]] = y[[0, 9, 10]] = gx[[0, 9, 10]] = gh[[0, 9, 10]] = np.nan
    out, h, e, eh = OB.block_norm(x, y, **kw)
    got = OB.block_norm_backward(gx, gh, np.where(np.isnan(x), np.nan, out), y, **kw)
    for a in (out, h, got["dx"][0], got["dy"][0]):
        assert np.isfinite(a).all() and (a[[0, 9, 10]] == 0).all()
    assert (e[[0, 9, 10]] == 0).all() and (eh[[0, 9, 10]] == 0).all() and (got["dgate"][0][1] == 0).all()


def test_bounds_hold_in_fp32_and_catch_mistakes():
    """An fp32 evaluation in numpy stays inside the bounds; a wrong formula does not."""
    x, y, gx, gh, kw = case(9, T=40, W=640, cu=(0, 13, 40))
    f = np.float32
    x, y, gx, gh = (v.astype(f) for v in (x, y, gx, gh))
    kw = {k: v.astype(f) if isinstance(v, np.ndarray) and k != "cu" else v for k, v in kw.items()}
    ro, rh, eo, eh = OB.block_norm(x, y, **kw)
    g = np.repeat(kw["gate"], [13, 27], 0)

    def fp32(eps=1e-5, a=0.9, mean=lambda v: (v * v).mean(1, keepdims=True, dtype=f), gate=g, pre=kw["pre_weight"]):
        n = y * (1 / np.sqrt(mean(y) + f(eps))) * kw["post_weight"]
        o = f(a) * x + f(0.4) * gate * n
        return o, o * (1 / np.sqrt(mean(o) + f(eps))) * pre
    o, h = fp32()
    assert OB.compare(o, ro, eo)["fails"] == 0 and OB.compare(h, rh, eh)["fails"] == 0
    for wrong in (dict(a=0.90001), dict(eps=1e-3), dict(gate=kw["gate"][:1]), dict(pre=kw["pre_weight"] * f(1.0001)),
                  dict(mean=lambda v: (v * v).sum(1, keepdims=True, dtype=f) / f(639))):
        o, h = fp32(**wrong)
        assert OB.compare(o, ro, eo)["fails"] + OB.compare(h, rh, eh)["fails"] > 0, wrong
