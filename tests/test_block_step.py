"""A whole transformer block's training step through the library: the first
norm, projection, query/key norm with a rotation by two axes, attention with
capped and biased scores behind prefixes, output projection, the norm behind
it with each sequence's gate and the next norm, a gated feed-forward with a
shared gate, the last norm, vocabulary projection and cross-entropy, and the
whole backward pass, every result against torch's float64 autograd of the same
step on the CPU.

The bound: each stage is good to some 1e-6 of its magnitudes (sums of at most
500 products and exponentials at 2^-24), and some twenty stages follow one
another, so gradients agree to 1e-4 in the 2-norm."""
import numpy as np
import pytest

from _gpu import say, to_dev

pytestmark = pytest.mark.gpu

HQ, HK, D, WIDTH, HIDDEN, VOCAB = 6, 2, 32, 192, 320, 500
CAP, RS, BS = 6.0, 0.8, 0.5
CU, PREFIX = [0, 1, 70, 70, 150], [0, 30, 5, 80]
T = 160                                        # ten rows of padding behind


def parameters():
    r = np.random.default_rng(0)
    f = lambda *s: r.standard_normal(s).astype(np.float32)  # noqa: E731
    w = lambda a, b: f(a, b) / np.float32(a ** 0.5)  # noqa: E731
    p = {"X": f(T, WIDTH), "Wqkv": w(WIDTH, (HQ + 2 * HK) * D), "Wo": w(HQ * D, WIDTH), "Wg": w(WIDTH, HIDDEN),
         "Wu": w(WIDTH, HIDDEN), "Wd": w(HIDDEN, WIDTH), "Wv": w(WIDTH, VOCAB), "gate1": 0.5 + 0.2 * f(4, WIDTH),
         "gate2": 0.5 + 0.2 * f(WIDTH), "slopes": 0.3 * 2.0 ** -np.arange(HQ, dtype=np.float32)}
    p.update({n: 1 + 0.1 * f(m) for n, m in (("qw", D), ("kw", D), ("w0", WIDTH), ("w1", WIDTH), ("w2", WIDTH),
                                             ("wp", WIDTH))})
    pos = r.integers(0, 40, (2, T)).astype(np.int32)
    axis = (np.arange(D // 2) % 2).astype(np.int32)
    freq = (100.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
    targets = r.integers(0, VOCAB, T).astype(np.int32)
    targets[CU[-1]:] = -1
    return p, pos, axis, freq, targets


def reference(p, pos, axis, freq, targets):
    import torch
    t = {n: torch.from_numpy(a).double().requires_grad_() for n, a in p.items()}
    norm = lambda x, w: x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
    total = 0.0
    for b, (s0, s1) in enumerate(zip(CU[:-1], CU[1:])):
        n = s1 - s0
        if n == 0:
            continue
        x = t["X"][s0:s1]
        q, k, v = (norm(x, t["w0"]) @ t["Wqkv"]).split([HQ * D, HK * D, HK * D], 1)
        angle = torch.from_numpy(pos[axis][:, s0:s1]).double().T * torch.from_numpy(freq).double()
        c, s = angle.cos()[:, None], angle.sin()[:, None]

        def turn(z, w):
            z = norm(z.reshape(n, -1, D), w)
            a, e = z[..., :D // 2], z[..., D // 2:]
            return torch.cat((a * c - e * s, e * c + a * s), -1)
        q, k = turn(q, t["qw"]), turn(k, t["kw"]).repeat_interleave(HQ // HK, 1)
        v = v.reshape(n, HK, D).repeat_interleave(HQ // HK, 1)
        i = torch.arange(n)
        away = (i[:, None] - i[None]).abs()
        sc = torch.einsum("ihd,jhd->hij", q, k) / D ** 0.5
        sc = CAP * torch.tanh(sc / CAP) - t["slopes"][:, None, None] * away
        see = (i[:, None] >= i[None]) | (i[None] < PREFIX[b])
        att = torch.einsum("hij,jhd->ihd", torch.softmax(sc.masked_fill(~see, -np.inf), -1), v).reshape(n, -1)
        x = RS * x + BS * t["gate1"][b] * norm(att @ t["Wo"], t["wp"])
        h = norm(x, t["w1"])
        x = x + t["gate2"] * ((torch.nn.functional.silu(h @ t["Wg"]) * (h @ t["Wu"])) @ t["Wd"])
        logits = norm(x, t["w2"]) @ t["Wv"]
        total = total - torch.log_softmax(logits, 1).gather(1, torch.from_numpy(targets[s0:s1]).long()[:, None]).sum()
    loss = total / CU[-1]
    loss.backward()
    return loss.item(), {n: x.grad.numpy() for n, x in t.items()}


def step(B, t, pos, axis, freq, targets, cu, prefix):
    import torch
    g = {}
    qk = (t["qw"], t["kw"], pos, freq)
    scores = {"cu_seqlens": cu, "softcap": CAP, "slopes": t["slopes"], "prefix_lens": prefix}
    first = {"pre_weight": t["w0"], "cu_seqlens": cu}
    middle = {"pre_weight": t["w1"], "post_weight": t["wp"], "gate": t["gate1"], "residual_scale": RS,
              "block_scale": BS, "cu_seqlens": cu}
    last = {"pre_weight": t["w2"], "gate": t["gate2"], "cu_seqlens": cu}
    split = lambda m: [x.unflatten(1, (-1, D)) for x in m.split([HQ * D, HK * D, HK * D], 1)]  # noqa: E731
    x0, h0 = B.block_norm(t["X"], **first)
    qkv = B.matmul(h0, t["Wqkv"])
    q0, k0, v = split(qkv)
    q, k = B.qk_norm_rope(q0, k0, *qk, pair_axis=axis)
    att, lse = B.attention(q, k, v, **scores)
    a = B.matmul(att.view(T, -1), t["Wo"])
    x1, h1 = B.block_norm(x0, a, **middle)
    gate, up = B.matmul(h1, t["Wg"]), B.matmul(h1, t["Wu"])
    y = B.matmul_residual_swiglu_a(gate, up, t["Wd"], torch.zeros_like(x1))
    x2, h2 = B.block_norm(x1, y, **last)
    logits = B.matmul(h2, t["Wv"])
    losses = B.cross_entropy(logits, targets, inv_norm=1.0 / CU[-1])

    g["Wv"] = B.matmul_at(h2, logits)                      # logits now holds their gradient
    dx, dy, g["w2"], _, g["gate2"] = B.block_norm_backward(None, B.matmul_t(logits, t["Wv"]), x2, y, **last)
    g["Wd"] = B.matmul_at_swiglu_a(gate, up, dy)
    dgate, dup = B.matmul_t_swiglu_backward(dy, t["Wd"], gate, up)
    g["Wg"], g["Wu"] = B.matmul_at(h1, dgate), B.matmul_at(h1, dup)
    dh = B.matmul_t(dgate, t["Wg"])
    B.matmul_t(dup, t["Wu"], out=dh, acc=True)
    dx, da, g["w1"], g["wp"], g["gate1"] = B.block_norm_backward(dx, dh, x1, a, **middle, dx=dx, dy=dh)
    g["Wo"] = B.matmul_at(att.view(T, -1), da)
    datt = B.matmul_t(da, t["Wo"]).view(T, HQ, D)
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = split(dqkv)
    g["slopes"] = torch.empty_like(t["slopes"])
    B.attention_backward(datt, q, k, v, att, lse, **scores, dq=dq, dk=dk, dv=dv, dslopes=g["slopes"])
    _, _, g["qw"], g["kw"] = B.qk_norm_rope_backward(dq, dk, q0, k0, *qk, pair_axis=axis, dq=dq, dk=dk)
    g["Wqkv"] = B.matmul_at(h0, dqkv)
    g["X"], _, g["w0"], _, _ = B.block_norm_backward(dx, B.matmul_t(dqkv, t["Wqkv"]), x0, **first, dx=dx)
    return B.sum_losses(losses), g


def test_block_step():
    import torch
    from tiled_dense_gemm_matmul_amd import binding as B
    p, pos, axis, freq, targets = parameters()
    want_loss, want = reference(p, pos, axis, freq, targets)
    t = {n: to_dev(a) for n, a in p.items()}
    args = [to_dev(x) for x in (pos, axis, freq, targets, np.array(CU, np.int32), np.array(PREFIX, np.int32))]
    loss, grads = step(B, t, *args)
    torch.cuda.synchronize()
    loss = loss.item() / CU[-1]
    say(f"block step: loss {loss:.6f}, reference {want_loss:.6f}")
    assert abs(loss - want_loss) < 5e-6 * abs(want_loss)
    assert set(grads) == set(want)
    for n, g in grads.items():
        far = np.linalg.norm(g.cpu().numpy() - want[n]) / np.linalg.norm(want[n])
        say(f"  {n}: {far:.2e}")
        assert far < 1e-4, (n, far)
    assert not bool(grads["X"][CU[-1]:].any())
    again, grads2 = step(B, t, *args)
    assert all(torch.equal(grads[n], grads2[n]) for n in grads) and again.item() / CU[-1] == loss
