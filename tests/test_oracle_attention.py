"""Pins of the attention and distillation oracles on the CPU: closed forms,
central differences of the forward definitions, and torch's float64 functions
where they compute the same thing."""
import numpy as np
import pytest

from oracle import attention as OA
from oracle import loss as OL


def _qkv(seed, T, hq, hk, d):
    r = np.random.default_rng(seed)
    return r.standard_normal((T, hq, d)), r.standard_normal((T, hk, d)), r.standard_normal((T, hk, d))


def test_one_key_returns_its_value():
    q, k, v = _qkv(0, 5, 2, 1, 8)
    out, lse, _, _ = OA.attention(q, k, v, window=1)
    np.testing.assert_allclose(out, np.repeat(v, 2, axis=1), rtol=1e-15)
    np.testing.assert_allclose(lse, (q * k).sum(2).T / np.sqrt(8), rtol=1e-13)


def test_equal_scores_average():
    q, k, v = _qkv(1, 6, 1, 1, 4)
    out, lse, _, _ = OA.attention(q * 0, k, v, causal=True)
    want = np.cumsum(v[:, 0], 0) / np.arange(1, 7)[:, None]
    np.testing.assert_allclose(out[:, 0], want, rtol=1e-14)
    np.testing.assert_allclose(lse[0], np.log(np.arange(1, 7)), atol=1e-14)


def test_rows_of_no_sequence():
    q, k, v = _qkv(2, 9, 2, 2, 4)
    out, lse, _, _ = OA.attention(q, k, v, cu=[2, 5, 5, 7])
    for rows in (slice(0, 2), slice(7, 9)):
        assert not out[rows].any() and np.all(lse[:, rows] == -np.inf)
    alone = OA.attention(q[5:7], k[5:7], v[5:7])
    np.testing.assert_array_equal(out[5:7], alone[0])


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 3), (False, 3)])
def test_attention_against_torch(causal, window):
    import torch
    q, k, v = _qkv(3, 11, 4, 2, 8)
    out, lse, _, _ = OA.attention(q, k, v, causal=causal, window=window)
    tq, tk, tv = (torch.from_numpy(x).transpose(0, 1) for x in (q, np.repeat(k, 2, 1), np.repeat(v, 2, 1)))
    s = (tq @ tk.transpose(1, 2)) / np.sqrt(8)
    s = s.masked_fill(~torch.from_numpy(OA.visible(11, causal, window)), -np.inf)
    np.testing.assert_allclose(out, (torch.softmax(s, -1) @ tv).transpose(0, 1).numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(lse, torch.logsumexp(s, -1).numpy(), rtol=1e-13)


def _differences(f, x, g, h=1e-5):
    """Central differences of sum(f(x) g) for every element of x."""
    d = np.zeros_like(x)
    flat, out = x.reshape(-1), d.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + h
        up = (f() * g).sum()
        flat[i] = keep - h
        down = (f() * g).sum()
        flat[i] = keep
        out[i] = (up - down) / (2 * h)
    return d


@pytest.mark.parametrize("causal,window,cu", [(True, 0, None), (False, 0, [1, 4, 7]), (True, 2, [0, 7]),
                                              (False, 3, None)])
def test_attention_backward_against_differences(causal, window, cu):
    q, k, v = _qkv(4, 7, 4, 2, 4)
    g = np.random.default_rng(5).standard_normal(q.shape)
    out, lse, _, _ = OA.attention(q, k, v, cu, causal, window)
    dq, dk, dv = OA.attention_backward(g, q, k, v, out, lse, cu, causal, window)[:3]
    f = lambda: OA.attention(q, k, v, cu, causal, window)[0]  # noqa: E731
    for got, x in ((dq, q), (dk, k), (dv, v)):
        np.testing.assert_allclose(got, _differences(f, x, g), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("rotated,interleaved", [(8, False), (8, True), (4, False), (4, True), (0, False)])
def test_norm_and_rotation(rotated, interleaved):
    r = np.random.default_rng(6)
    x, w = r.standard_normal((3, 2, 8)), 1 + 0.1 * r.standard_normal(8)
    pos, freq = np.array([0, 5, -3]), 100.0 ** (-np.arange(rotated // 2) / max(1, rotated // 2))
    y, _ = OA.qk_norm_rope(x, w, pos, freq, 1e-6, interleaved)
    n = x / np.sqrt((x * x).mean(2, keepdims=True) + 1e-6) * w
    np.testing.assert_allclose(y[0], n[0], rtol=1e-14)  # position 0 turns nothing
    np.testing.assert_allclose(y[..., rotated:], n[..., rotated:], rtol=1e-14)
    np.testing.assert_allclose((y * y).sum(2), (n * n).sum(2), rtol=1e-13)  # a rotation
    if rotated:
        a, b = (0, 1) if interleaved else (0, rotated // 2)  # pair 0 turns by pos * 1
        z = (n[1, :, a] + 1j * n[1, :, b]) * np.exp(5j)
        np.testing.assert_allclose(y[1, :, a] + 1j * y[1, :, b], z, rtol=1e-13)
    g = r.standard_normal(x.shape)
    dx, dw, _, _ = OA.qk_norm_rope_backward(g, x, w, pos, freq, 1e-6, interleaved)
    f = lambda: OA.qk_norm_rope(x, w, pos, freq, 1e-6, interleaved)[0]  # noqa: E731
    np.testing.assert_allclose(dx, _differences(f, x, g), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dw, _differences(f, w, g), rtol=1e-6, atol=1e-8)


def _distill_case(seed, S=5, V=12, K=4):
    r = np.random.default_rng(seed)
    ids = r.integers(0, V, (S, K))
    ids[1, 2] = ids[1, 0]      # one column twice
    ids[2, 1] = -1             # an unused entry
    ids[3] = V                 # a row without a teacher
    z = r.standard_normal((S, K)) * 2
    z[2, 1] = np.nan
    t = r.integers(0, V, S)
    t[1] = ids[1, 0]           # the target among the teacher's columns
    t[4] = -1                  # padding
    return r.standard_normal((S, V)) * 2, t, ids, z


@pytest.mark.parametrize("tau,mix,alpha,beta", [(1.0, 0.5, 0.0, 0.0), (2.5, 0.3, 0.1, 1e-2), (0.7, 1.0, 0.0, 0.0)])
def test_distill_against_differences(tau, mix, alpha, beta):
    l, t, ids, z = _distill_case(7)
    losses, dl, _ = OL.distill(l, t, ids, z, tau, mix, alpha, beta, 0.25)
    assert not dl[4].any() and not losses[:, 4].any() and losses[1, 3] == 0.0

    def total():
        a = OL.distill(l, t, ids, z, tau, mix, alpha, beta, 0.25)[0]
        return (1 - mix) * a[0] + mix * a[1]
    np.testing.assert_allclose(dl, _differences(total, l, np.full(5, 0.25)), rtol=1e-6, atol=1e-9)


def test_distill_is_a_divergence():
    """Zero exactly where the student has the teacher's distribution, and the
    plain cross-entropy gradient for a teacher that is sure of the target."""
    l = np.log(np.array([[0.2, 0.3, 0.5]]))
    ids, z = np.array([[2, 0, 1]]), np.log(np.array([[0.5, 0.2, 0.3]])) + 4.0
    losses, dl, _ = OL.distill(l, None, ids, z, 1.0, 1.0)
    assert abs(losses[1, 0]) < 1e-15 and np.abs(dl).max() < 1e-15
    r = np.random.default_rng(8)
    l = r.standard_normal((3, 9))
    t = np.array([4, 0, 8])
    one, g1, _ = OL.distill(l, None, t[:, None], np.zeros((3, 1)), 1.0, 1.0)
    two, g2, _ = OL.cross_entropy(l, t)
    np.testing.assert_allclose(one[1], two, rtol=1e-13)
    np.testing.assert_allclose(g1, g2, rtol=1e-12, atol=1e-15)
