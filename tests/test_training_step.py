"""A transformer block's training step through the library from end to end:
projection, query/key norm and rotation, attention over packed sequences,
output projection with the residual, vocabulary projection, distillation
loss, and the whole backward pass, every result against torch's float64
autograd of the same step on the CPU.

The bound: each of the chain's stages is good to some 1e-6 of its magnitudes
(sums of at most 500 products and exponentials at 2^-24), and a dozen
stages follow one another, so gradients agree to 5e-5 in the 2-norm."""
import numpy as np
import pytest

from _gpu import device, say, to_dev

pytestmark = pytest.mark.gpu


def reference(p, cu, ids, z, targets, pos, freq, hq, hk, d, tau, mix, window):
    import torch
    t = {n: torch.from_numpy(a).double().requires_grad_() for n, a in p.items()}
    T = p["X"].shape[0]
    rows = slice(cu[0], cu[-1])
    qkv = t["X"] @ t["Wqkv"]
    q, k, v = qkv.split([hq * d, hk * d, hk * d], 1)
    angle = torch.outer(torch.from_numpy(pos).double(), torch.from_numpy(freq).double())
    c, s = angle.cos()[:, None], angle.sin()[:, None]

    def norm(x, w):
        x = x.view(T, -1, d)
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        a, b = x[..., :d // 2], x[..., d // 2:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)
    q, k, v = norm(q, t["qw"]), norm(k, t["kw"]), v.view(T, hk, d)
    k, v = (x.repeat_interleave(hq // hk, 1) for x in (k, v))
    parts = [torch.zeros(cu[0], hq, d, dtype=torch.float64)]
    for a, b in zip(cu[:-1], cu[1:]):
        i = torch.arange(b - a)
        see = (i[:, None] >= i[None]) & (i[:, None] - i[None] < window)
        sc = torch.einsum("ihd,jhd->hij", q[a:b], k[a:b]) / d ** 0.5
        parts.append(torch.einsum("hij,jhd->ihd", torch.softmax(sc.masked_fill(~see, -np.inf), -1), v[a:b]))
    parts.append(torch.zeros(T - cu[-1], hq, d, dtype=torch.float64))
    y = torch.cat(parts).reshape(T, -1) @ t["Wo"] + t["X"]
    logits = y @ t["Wv"]
    real = torch.from_numpy(targets).long()
    keep = torch.from_numpy((targets >= 0).astype(float))
    ce = -torch.log_softmax(logits, 1).gather(1, real.clamp(min=0)[:, None])[:, 0]
    share = torch.log_softmax(torch.from_numpy(z).double() / tau, 1)
    far = share - torch.log_softmax(logits / tau, 1).gather(1, torch.from_numpy(ids).long())
    kd = tau ** 2 * (share.exp() * far).sum(1)
    loss = (keep * ((1 - mix) * ce + mix * kd)).sum() / keep.sum()
    loss.backward()
    assert rows.stop <= T
    return loss.item(), {n: x.grad.numpy() for n, x in t.items()}


def test_block_step():
    import torch
    from tiled_dense_gemm_matmul_amd import binding as B
    hq, hk, d, width, vocab, K, tau, mix, window = 6, 2, 32, 192, 500, 16, 2.0, 0.6, 50
    cu = [0, 1, 70, 70, 150]
    T = 160                                    # ten rows of padding behind
    r = np.random.default_rng(0)
    f = lambda *s: r.standard_normal(s).astype(np.float32)  # noqa: E731
    p = {"X": f(T, width), "Wqkv": f(width, (hq + 2 * hk) * d) / np.float32(width ** 0.5),
         "Wo": f(hq * d, width) / np.float32((hq * d) ** 0.5), "Wv": f(width, vocab) / np.float32(width ** 0.5),
         "qw": 1 + 0.1 * f(d), "kw": 1 + 0.1 * f(d)}
    pos = np.concatenate([np.arange(b - a) for a, b in zip([*cu[:-1], cu[-1]], [*cu[1:], T])]).astype(np.int32)
    freq = (100.0 ** (-np.arange(d // 2) / (d // 2))).astype(np.float32)
    targets = r.integers(0, vocab, T).astype(np.int32)
    targets[cu[-1]:] = -1
    ids = np.stack([r.permutation(vocab)[:K] for _ in range(T)]).astype(np.int32)
    z = f(T, K) * 2
    want_loss, want = reference(p, cu, ids, z, targets, pos, freq, hq, hk, d, tau, mix, window)

    t = {n: to_dev(a) for n, a in p.items()}
    dcu, dpos, dfreq = to_dev(np.array(cu, np.int32)), to_dev(pos), to_dev(freq)
    split = lambda m: [x.unflatten(1, (-1, d)) for x in m.split([hq * d, hk * d, hk * d], 1)]  # noqa: E731
    norm = (t["qw"], t["kw"], dpos, dfreq)
    qkv = B.matmul(t["X"], t["Wqkv"])
    q0, k0, v = split(qkv)
    q, k = B.qk_norm_rope(q0, k0, *norm)
    att, lse = B.attention(q, k, v, cu_seqlens=dcu, window=window)
    y = B.matmul_residual(att.view(T, -1), t["Wo"], t["X"])
    logits = B.matmul(y, t["Wv"])
    losses = B.distill_cross_entropy(logits, to_dev(targets), to_dev(ids), to_dev(z), tau, mix)
    kept = int((targets >= 0).sum())
    loss = ((1 - mix) * B.sum_losses(losses[0]) + mix * B.sum_losses(losses[1])).item() / kept
    grads = {"Wv": B.matmul_at(y, logits)}                 # logits now holds their gradient
    dy = B.matmul_t(logits, t["Wv"])
    grads["Wo"] = B.matmul_at(att.view(T, -1), dy)
    datt = B.matmul_t(dy, t["Wo"]).view(T, hq, d)
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = split(dqkv)
    B.attention_backward(datt, q, k, v, att, lse, cu_seqlens=dcu, window=window, dq=dq, dk=dk, dv=dv)
    _, _, grads["qw"], grads["kw"] = B.qk_norm_rope_backward(dq, dk, q0, k0, *norm, dq=dq, dk=dk)
    grads["Wqkv"] = B.matmul_at(t["X"], dqkv)
    grads["X"] = B.matmul_t(dqkv, t["Wqkv"], out=dy, acc=True)   # the residual's gradient is there already
    torch.cuda.synchronize()
    say(f"block step: loss {loss:.6f}, reference {want_loss:.6f}")
    assert abs(loss - want_loss) < 5e-6 * abs(want_loss)
    for n, g in grads.items():
        far = np.linalg.norm(g.cpu().numpy() - want[n]) / np.linalg.norm(want[n])
        say(f"  {n}: {far:.2e}")
        assert far < 5e-5, (n, far)
    assert device() == logits.device
