"""Pins of the oracle of capped, biased and prefix-masked attention (CPU):
torch's float64 autograd written from the definition, the plain oracle where
the forms agree, closed forms, and planted mistakes."""
import numpy as np
import pytest

from oracle import attention as OA


def case(seed=0, lengths=(1, 7, 0, 5), first=2, tail=1, hq=4, hk=2, d=6):
    r = np.random.default_rng(seed)
    T = first + sum(lengths) + tail
    cu = np.cumsum([first, *lengths])
    q, k, v, g = (r.standard_normal((T, h, d)) for h in (hq, hk, hk, hq))
    return 3 * q, k, v, g, cu


FORMS = [dict(softcap=2.0), dict(slopes=[0.5, 0.1, -0.2, 0.0]), dict(prefix=[1, 4, 9, -3]), dict(prefix=[0, 100, 0, 2]),
         dict(softcap=1.5, slopes=[0.5, 0.1, 0.2, 0.3], prefix=[0, 3, 0, 4]),
         dict(softcap=5.0, slopes=[0.5, 0.1, 0.2, 0.3], window=3, prefix=[0, 6, 0, 4]),
         dict(softcap=5.0, slopes=[0.5, 0.1, 0.2, 0.3], window=2, causal=False)]


def by_definition(q, k, v, cu, causal=True, window=0, softcap=0.0, slopes=None, prefix=None):
    """One row at a time."""
    import torch
    T, hq, d = q.shape
    out, lse = [], []
    for i in range(T):
        b = next((b for b in range(len(cu) - 1) if cu[b] <= i < cu[b + 1]), None)
        for h in range(hq):
            if b is None:
                out.append(torch.zeros(d, dtype=torch.float64))
                lse.append(torch.tensor(-np.inf, dtype=torch.float64))
                continue
            scores, vals = [], []
            for j in range(cu[b], cu[b + 1]):
                if causal and j > i and not (prefix is not None and j - cu[b] < prefix[b]):
                    continue
                if window and abs(i - j) >= window:
                    continue
                s = (q[i, h] * k[j, h // (hq // k.shape[1])]).sum() / d ** 0.5
                if softcap:
                    s = softcap * torch.tanh(s / softcap)
                if slopes is not None:
                    s = s - slopes[h] * abs(i - j)
                scores.append(s)
                vals.append(v[j, h // (hq // k.shape[1])])
            scores = torch.stack(scores)
            lse.append(torch.logsumexp(scores, 0))
            out.append((torch.softmax(scores, 0)[:, None] * torch.stack(vals)).sum(0))
    return torch.stack(out).view(T, hq, d), torch.stack(lse).view(T, hq).t()


@pytest.mark.parametrize("form", FORMS)
def test_against_autograd(form):
    import torch
    q, k, v, g, cu = case()
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v)]
    sl = None if "slopes" not in form else torch.tensor(np.array(form["slopes"], dtype=float), requires_grad=True)
    out, lse = by_definition(*t, cu, **dict(form, slopes=sl))
    ro, rl, _, _ = OA.scored_attention(q, k, v, cu, **form)
    assert np.allclose(ro, out.detach().numpy(), rtol=1e-12, atol=1e-13)
    used = np.isfinite(rl)
    assert np.array_equal(used, np.isfinite(lse.detach().numpy())) and np.allclose(rl[used], lse.detach().numpy()[used])
    (out * torch.tensor(g)).sum().backward()
    got = OA.scored_attention_backward(g, q, k, v, ro, rl, cu, **form)
    for x, y in zip(got, t):
        assert np.allclose(x, y.grad.numpy(), rtol=1e-10, atol=1e-12)
    if sl is not None:
        assert np.allclose(got[3], sl.grad.numpy(), rtol=1e-10, atol=1e-12)
    assert all((e >= 0).all() for e in got[4:])


def test_plain_scores_are_the_plain_oracle():
    q, k, v, g, cu = case(3)
    for kw in (dict(), dict(window=3), dict(causal=False)):
        a, b = OA.attention(q, k, v, cu, **kw), OA.scored_attention(q, k, v, cu, **kw)
        assert np.allclose(a[0], b[0]) and np.array_equal(np.isfinite(a[1]), np.isfinite(b[1]))
        x, y = (f(g, q, k, v, a[0], a[1], cu, **kw) for f in (OA.attention_backward, OA.scored_attention_backward))
        assert all(np.allclose(i, j) for i, j in zip(x[:3], y[:3]))
    a = OA.attention(q, k, v, cu, causal=False)
    b = OA.scored_attention(q, k, v, cu, prefix=[99] * 4)  # a prefix as long as the sequence hides nothing
    assert np.allclose(a[0], b[0])


def test_closed_forms():
    """Equal keys under a slope: a geometric series; a cap that all scores reach: the mean."""
    q, k = np.ones((9, 1, 4)), np.ones((9, 1, 4))
    v = np.arange(9.0)[:, None, None] * np.ones((9, 1, 4))
    out = OA.scored_attention(q, k, v, slopes=[np.log(2.0)])[0]
    w = 0.5 ** np.arange(9)[::-1]
    assert np.allclose(out[8, 0], (w * np.arange(9)).sum() / w.sum())
    r = np.random.default_rng(0)
    k = 1e6 * np.abs(r.standard_normal((9, 1, 4)))
    assert np.allclose(OA.scored_attention(q, k, v, softcap=3.0, causal=False)[0], 4.0)


def test_visible():
    see = OA.scored_visible(5, True, 0, 3)
    want = np.tril(np.ones((5, 5), bool))
    want[:, :3] = True
    assert np.array_equal(see, want)
    assert np.array_equal(OA.scored_visible(5, True, 2, 3), want & (np.abs(np.subtract.outer(range(5), range(5))) < 2))


@pytest.mark.parametrize("wrong", [dict(softcap=2.001), dict(slopes=[0.5, 0.1, 0.2, 0.3001]), dict(prefix=[0, 4, 0, 4]),
                                   dict(softcap=0.0)])
def test_the_bounds_catch_mistakes(wrong):
    form = dict(softcap=2.0, slopes=[0.5, 0.1, 0.2, 0.3], prefix=[0, 3, 0, 4])
    q, k, v, g, cu = case(5)
    ro, rl, eo, el = OA.scored_attention(q, k, v, cu, **form)
    want = OA.scored_attention_backward(g, q, k, v, ro, rl, cu, **form)
    bad = OA.scored_attention(q, k, v, cu, **{**form, **wrong})
    assert OA.compare(bad[0], ro, eo)["fails"] and OA.compare(bad[1], rl, el)["fails"]
    got = OA.scored_attention_backward(g, q, k, v, ro, rl, cu, **{**form, **wrong})
    assert all(OA.compare(got[i], want[i], want[4 + i])["fails"] for i in range(4))


def test_an_fp32_evaluation_stays_inside_the_bounds():
    import torch
    form = dict(softcap=4.0, slopes=np.float32([0.5, 0.1, 0.2, 0.3]), prefix=[0, 3, 0, 4])
    q, k, v, g, cu = case(6)
    q, k, v, g = (x.astype(np.float32) for x in (q, k, v, g))
    ro, rl, eo, el = OA.scored_attention(q, k, v, cu, **form)
    T, hq, d = q.shape
    for b in range(4):
        a, e = cu[b], cu[b + 1]
        see = torch.tensor(OA.scored_visible(e - a, True, 0, form["prefix"][b]))
        for h in range(hq if e > a else 0):
            x, y, z = (torch.tensor(t[a:e, i]) for t, i in ((q, h), (k, h // 2), (v, h // 2)))
            i = torch.arange(e - a, dtype=torch.float32)
            s = 4.0 * torch.tanh(x @ y.T * np.float32(d ** -0.5) / 4.0) - float(form["slopes"][h]) * (i[:, None] - i).abs()
            p = torch.softmax(s.masked_fill(~see, -np.inf), 1)
            assert OA.compare((p @ z).numpy(), ro[a:e, h], eo[a:e, h])["fails"] == 0


def test_the_cap_keeps_its_derivative_where_it_saturates():
    """1 - tanh^2 is 4 e / (1 + e)^2, e = exp(-2 |x|): far below what is left of 1 - t t in 64 bits, and not zero.
    A row that sees one key alone has ds = 0, which fp32 forms to some roundings of dout . v; times that derivative
    they are what dq may be off by."""
    from decimal import Decimal
    for x in (0.0, 0.3, -2.0, 9.0, 18.0, -19.5, 25.0, 100.0, 300.0):
        steep = OA._final_scores(np.array([[x]]), np.array([[1.0]]), 1.0, 1.0, 0.0)[1][0, 0]
        e = (Decimal(-2) * abs(Decimal(x))).exp()
        assert abs(Decimal(steep) / (4 * e / (1 + e) ** 2) - 1) < Decimal(1e-13), x
    assert OA._final_scores(np.array([[1e30]]), np.array([[1.0]]), 1.0, 1.0, 0.0)[1][0, 0] < 1e-300
    q, k, v, g = np.full((1, 1, 4), 12.5), np.ones((1, 1, 4)), np.full((1, 1, 4), 0.5), np.ones((1, 1, 4))
    out, lse, _, _ = OA.scored_attention(q, k, v, softcap=1.0)
    dq, _, _, _, e_dq = OA.scored_attention_backward(g, q, k, v, out, lse, softcap=1.0)[:5]
    # ds of three roundings of dout . v = 2, the derivative at x = 25, scale 1/2
    assert not dq.any() and (e_dq > 0.5 * 4 * np.exp(-50.0) * 3 * 2.0 ** -24 * 2).all() and (e_dq < 1e-25).all()


@pytest.mark.parametrize("axes", [1, 3])
def test_far_positions_without_a_rotated_pair(axes):
    """Heads that are normed and not turned, at positions of any size."""
    r = np.random.default_rng(0)
    x, w, pos = r.standard_normal((5, 2, 8)), r.standard_normal(8), np.full((axes, 5), 1 << 50)
    y = OA.qk_norm_rope(x, w, pos, np.zeros(0), axis=np.zeros(0, np.int32))[0]
    assert np.array_equal(y, OA.qk_norm_rope(x, w, pos[0] * 0, np.zeros(0))[0])
