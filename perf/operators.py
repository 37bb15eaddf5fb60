"""The operators around the linear layers of a training step, as they are measured: attention over packed sequences
and its backward pass, the per-head norm of queries and keys with the position rotation and its backward pass, and
cross-entropy with distillation from a teacher's top logits.

`own` False computes each operator in its plain form with elementary torch operations; `own` True makes the calls a
user makes of tiled_dense_gemm_matmul_amd.binding.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"


def listed():
    return [
        # one short prompt through the 768-wide model's 12 heads: launch latency counts
        {"name": "attention_short", "op": "attention", "lengths": "77", "tail": 0, "q_heads": 12, "kv_heads": 12,
         "dim": 64, "causal": True, "window": 0},
        # the 16 x 512-token batch of that model
        {"name": "attention_batch16x512", "op": "attention", "lengths": ",".join(["512"] * 16), "tail": 0,
         "q_heads": 12, "kv_heads": 12, "dim": 64, "causal": True, "window": 0},
        # documents of very different lengths packed into one buffer, shared heads, a sliding window, unused rows behind
        {"name": "attention_packed_window", "op": "attention", "lengths": "1,613,2047,33,4096,130,999", "tail": 73,
         "q_heads": 16, "kv_heads": 4, "dim": 128, "causal": True, "window": 1000},
        # one sequence of 512 tokens, the model's training length
        {"name": "attention_backward_seq512", "op": "attention_backward", "lengths": "512", "tail": 0, "q_heads": 12,
         "kv_heads": 12, "dim": 64, "causal": True, "window": 0},
        # one long document with shared heads
        {"name": "attention_backward_long", "op": "attention_backward", "lengths": "8191", "tail": 0, "q_heads": 12,
         "kv_heads": 4, "dim": 64, "causal": True, "window": 0},
        # packed documents that look both ways (an encoder's), heads as wide as 128
        {"name": "attention_backward_packed", "op": "attention_backward", "lengths": "700,1,1531,257,64,1200",
         "tail": 31, "q_heads": 8, "kv_heads": 2, "dim": 128, "causal": False, "window": 0},
        # one 512-token sequence of the 768-wide model, between its projections and attention
        {"name": "qk_norm_rope_seq512", "op": "qk_norm_rope", "tokens": 512, "q_heads": 12, "kv_heads": 12, "dim": 64,
         "rotated": 64, "interleaved": False, "first": 0, "wide_positions": False},
        # 8192 tokens of a wider model with shared heads, late in a long document
        {"name": "qk_norm_rope_8192", "op": "qk_norm_rope", "tokens": 8192, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rotated": 128, "interleaved": False, "first": 120000, "wide_positions": True},
        # an odd number of tokens, part of each head rotated in neighbouring pairs
        {"name": "qk_norm_rope_backward_odd", "op": "qk_norm_rope_backward", "tokens": 1001, "q_heads": 6,
         "kv_heads": 2, "dim": 96, "rotated": 32, "interleaved": True, "first": 0, "wide_positions": False},
        # the 16 x 512-token batch of the 768-wide model
        {"name": "qk_norm_rope_backward_8192", "op": "qk_norm_rope_backward", "tokens": 8192, "q_heads": 12,
         "kv_heads": 12, "dim": 64, "rotated": 64, "interleaved": False, "first": 0, "wide_positions": True},
        # the seq-512 model's logits against a teacher's 64 best, stored in 16 bits
        {"name": "distill_512x16384", "op": "distill", "rows": 512, "vocab": 16384, "top": 64, "half": True,
         "wide_ids": False, "temperature": 2.0, "mix": 0.5, "alpha": 0.0, "beta": 0.0},
        # a batch of 4093 rows over an odd vocabulary, with label smoothing and z-loss in the hard term
        {"name": "distill_4093x50257", "op": "distill", "rows": 4093, "vocab": 50257, "top": 100, "half": False,
         "wide_ids": True, "temperature": 1.0, "mix": 0.7, "alpha": 0.1, "beta": 1e-4},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["attention", "attention_backward", "qk_norm_rope", "qk_norm_rope_backward", "distill"])
    if op.startswith("attention"):
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4])
        dim = rng.choice([32, 48, 64, 80, 96, 128])
        lengths = [_log_int(rng, 1, 4096) for _ in range(_log_int(rng, 1, 16))]
        # the padded scores of the plain form stay below those of the largest listed case
        while len(lengths) * heads * dim * max(lengths) ** 2 > 2 ** 35 or sum(lengths) > 8192:
            lengths[lengths.index(max(lengths))] = max(1, max(lengths) * 2 // 3)
        window = rng.choice([0, 0, _log_int(rng, 1, 2000)])
        return {"op": op, "lengths": ",".join(map(str, lengths)), "tail": rng.choice([0, rng.randrange(100)]),
                "q_heads": heads, "kv_heads": kv, "dim": dim, "causal": rng.random() < 0.75, "window": window}
    if op.startswith("qk_norm_rope"):
        kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([32, 64, 96, 128])
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "q_heads": kv * rng.choice([1, 2, 3, 4]), "kv_heads": kv,
                "dim": dim, "rotated": rng.choice([dim, dim // 2, 16]), "interleaved": rng.random() < 0.5,
                "first": rng.choice([0, rng.randrange(1000000)]), "wide_positions": rng.random() < 0.5}
    vocab = _log_int(rng, 300, 70000)
    return {"op": op, "rows": _log_int(rng, 1, max(1, min(8192, 200000000 // vocab))), "vocab": vocab,
            "top": _log_int(rng, 1, 200), "half": rng.random() < 0.5, "wide_ids": rng.random() < 0.5,
            "temperature": rng.choice([1.0, round(rng.uniform(0.5, 4.0), 3)]), "mix": rng.choice([1.0, 0.5, 0.9]),
            "alpha": rng.choice([0.0, 0.1]), "beta": rng.choice([0.0, 1e-4])}


# --- what a user's program has in hand ---


def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEVICE)

    if case["op"].startswith("attention"):
        return _prepare_attention(case, normal)
    if case["op"].startswith("qk_norm_rope"):
        return _prepare_qk(case, normal)
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    logits = normal(rows, vocab) * 3.0
    targets = torch.randint(vocab, (rows,), generator=g, device=DEVICE, dtype=torch.int32)
    targets[16::17] = -1  # padding rows
    ids = torch.randint(vocab, (rows, top), generator=g, device=DEVICE, dtype=torch.int64)
    ids[:, top // 2 + 1:][torch.rand((rows, top - top // 2 - 1), generator=g, device=DEVICE) < 0.1] = -1  # unused slots
    z = normal(rows, top) * 2.0 + 8.0
    return {"case": case, "logits": logits, "targets": targets, "ids": ids if case["wide_ids"] else ids.int(),
            "teacher": z.half() if case["half"] else z, "inv_norm": 1.0 / max(1, rows - rows // 17),
            "dlogits": torch.empty_like(logits)}


def _prepare_attention(case, normal):
    lengths = _lengths(case)
    tokens = sum(lengths) + case["tail"]
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    # queries, keys and values as one projection writes them
    qkv = normal(tokens, (hq + 2 * hkv) * dim)
    q, k, v = qkv.split([hq * dim, hkv * dim, hkv * dim], dim=1)
    state = {"case": case, "q": q.view(tokens, hq, dim), "k": k.view(tokens, hkv, dim), "v": v.view(tokens, hkv, dim),
             "cu_seqlens": torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32, device=DEVICE),
             "longest": max(lengths)}
    if case["op"] == "attention_backward":
        state["out"], state["lse"] = _attention(state)
        state["dout"] = normal(tokens, hq, dim)
    return state


def _prepare_qk(case, normal):
    tokens, hq, hkv, dim = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    qkv = normal(tokens, (hq + 2 * hkv) * dim)
    state = {"case": case, "q": qkv[:, :hq * dim].view(tokens, hq, dim),
             "k": qkv[:, hq * dim:(hq + hkv) * dim].view(tokens, hkv, dim),
             "q_weight": 1.0 + 0.1 * normal(dim), "k_weight": 1.0 + 0.1 * normal(dim),
             "positions": case["first"] + torch.arange(tokens, device=DEVICE,
                                                       dtype=torch.int64 if case["wide_positions"] else torch.int32),
             "inv_freq": torch.tensor(10000.0 ** (-np.arange(0, case["rotated"], 2) / case["rotated"]),
                                      dtype=torch.float32, device=DEVICE)}
    if case["op"] == "qk_norm_rope_backward":
        state["dq_out"], state["dk_out"] = normal(tokens, hq, dim), normal(tokens, hkv, dim)
    return state


# --- one pass ---


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_attention(s):
    from tiled_dense_gemm_matmul_amd import binding
    return binding.attention(s["q"], s["k"], s["v"], cu_seqlens=s["cu_seqlens"], causal=s["case"]["causal"],
                             window=s["case"]["window"])


def _own_attention_backward(s):
    from tiled_dense_gemm_matmul_amd import binding
    return binding.attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"],
                                      cu_seqlens=s["cu_seqlens"], causal=s["case"]["causal"],
                                      window=s["case"]["window"])


def _own_qk_norm_rope(s):
    from tiled_dense_gemm_matmul_amd import binding
    return binding.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"], eps=1e-6,
                                interleaved=s["case"]["interleaved"])


def _own_qk_norm_rope_backward(s):
    from tiled_dense_gemm_matmul_amd import binding
    return binding.qk_norm_rope_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["q_weight"], s["k_weight"],
                                         s["positions"], s["inv_freq"], eps=1e-6,
                                         interleaved=s["case"]["interleaved"])


def _own_distill(s):
    from tiled_dense_gemm_matmul_amd import binding
    c = s["case"]
    losses = binding.distill_cross_entropy(s["logits"], s["targets"], s["ids"], s["teacher"],
                                           temperature=c["temperature"], mix=c["mix"], alpha=c["alpha"],
                                           beta=c["beta"], inv_norm=s["inv_norm"], dlogits=s["dlogits"])
    return losses, s["dlogits"]


_OWN = {"attention": _own_attention, "attention_backward": _own_attention_backward,
        "qk_norm_rope": _own_qk_norm_rope, "qk_norm_rope_backward": _own_qk_norm_rope_backward,
        "distill": _own_distill}


# --- the plain forms ---


class _Packing:
    """The padded batch [sequences, longest] of a packed buffer and the way back."""

    def __init__(self, s):
        c, cu, tokens = s["case"], s["cu_seqlens"].long(), s["q"].shape[0]
        start, length = cu[:-1], cu[1:] - cu[:-1]
        pos = torch.arange(s["longest"], device=cu.device)
        inside = pos[None, :] < length[:, None]
        self.index = torch.where(inside, start[:, None] + pos[None, :], 0)
        gap = pos[:, None] - pos[None, :]
        sees = (gap >= 0) if c["causal"] else torch.ones_like(gap, dtype=torch.bool)
        if c["window"]:
            sees = sees & (gap.abs() < c["window"])
        self.mask = (inside[:, :, None] & inside[:, None, :] & sees)[:, None, None]
        row = torch.arange(tokens, device=cu.device)
        self.seq = (row[:, None] >= cu[None, 1:]).sum(1).clamp(max=len(start) - 1)
        self.pos = (row - start[self.seq]).clamp(0, s["longest"] - 1)
        self.used = (row >= cu[0]) & (row < cu[-1])

    def pad(self, x, groups=1):
        """[tokens, heads, dim] to [sequences, heads / groups, groups * longest, dim]."""
        y = x[self.index].permute(0, 2, 1, 3)
        return y.reshape(y.shape[0], y.shape[1] // groups, -1, y.shape[3])

    def unpad(self, y, heads, empty=0.0):
        """[sequences, heads / groups, groups * longest, dim] to [tokens, heads, dim]."""
        y = y.reshape(y.shape[0], heads, -1, y.shape[-1])[self.seq, :, self.pos]
        return torch.where(self.used[:, None, None], y, empty)


def _scores(p, q, k, groups, scale):
    b, hkv, rows, _ = q.shape
    s = torch.matmul(q, k.transpose(2, 3)).mul_(scale).view(b, hkv, groups, rows // groups, k.shape[2])
    return s.masked_fill_(~p.mask, -math.inf)


def _attention(s):
    q, k, v = s["q"], s["k"], s["v"]
    heads, groups, p = q.shape[1], q.shape[1] // k.shape[1], _Packing(s)
    scores = _scores(p, p.pad(q, groups), p.pad(k), groups, q.shape[2] ** -0.5)
    top = scores.amax(-1, keepdim=True).clamp_(min=-3e38)
    probs = torch.exp(scores - top)
    total = probs.sum(-1, keepdim=True)
    probs = (probs / total.clamp(min=1e-30)).flatten(2, 3)
    out = p.unpad(torch.matmul(probs, p.pad(v)), heads)
    lse = p.unpad((top + torch.log(total)).flatten(2, 3), heads, -math.inf)
    return out, lse[:, :, 0].t().contiguous()


def _attention_backward(s):
    q, k, v = s["q"], s["k"], s["v"]
    heads, kv_heads, scale, p = q.shape[1], k.shape[1], q.shape[2] ** -0.5, _Packing(s)
    groups = heads // kv_heads
    qp, kp, vp, dp = p.pad(q, groups), p.pad(k), p.pad(v), p.pad(s["dout"], groups)
    lse = p.pad(s["lse"].t()[:, :, None], groups)
    delta = p.pad((s["dout"] * s["out"]).sum(-1, keepdim=True), groups)
    probs = torch.exp(_scores(p, qp, kp, groups, scale).flatten(2, 3) - lse)
    ds = probs * (torch.matmul(dp, vp.transpose(2, 3)) - delta)
    dq = torch.matmul(ds, kp) * scale
    dk = torch.matmul(ds.transpose(2, 3), qp) * scale
    dv = torch.matmul(probs.transpose(2, 3), dp)
    return p.unpad(dq, heads), p.unpad(dk, kv_heads), p.unpad(dv, kv_heads)


def _cos_sin(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]  # far positions need 64 bits
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _halves(x, rotated, interleaved):
    """The two members of each rotated pair, and what is not rotated."""
    y, rest = x[..., :rotated], x[..., rotated:]
    if interleaved:
        return y[..., 0::2], y[..., 1::2], rest
    return y[..., :rotated // 2], y[..., rotated // 2:], rest


def _join(a, b, rest, interleaved):
    pair = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((pair, rest), -1)


def _qk_norm_rope(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    result = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        a, b, rest = _halves(y, c["rotated"], c["interleaved"])
        result.append(_join(a * cos - b * sin, b * cos + a * sin, rest, c["interleaved"]))
    return result[0], result[1]


def _qk_norm_rope_backward(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    grads, weights = [], []
    for dy, x, w in ((s["dq_out"], s["q"], s["q_weight"]), (s["dk_out"], s["k"], s["k_weight"])):
        a, b, rest = _halves(dy, c["rotated"], c["interleaved"])
        dn = _join(a * cos + b * sin, b * cos - a * sin, rest, c["interleaved"])
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        n = x * r
        g = dn * w
        grads.append(r * (g - n * (g * n).mean(-1, keepdim=True)))
        weights.append((dn * n).sum((0, 1), dtype=torch.float64).float())  # a long sum
    return grads[0], grads[1], weights[0], weights[1]


def _distill(s):
    c, logits, inv_norm = s["case"], s["logits"], s["inv_norm"]
    tau, mix, alpha, beta = c["temperature"], c["mix"], c["alpha"], c["beta"]
    vocab = logits.shape[1]
    target, ids = s["targets"].long(), s["ids"].long()
    kept = ((target >= 0) & (target < vocab))[:, None]
    target = target.clamp(0, vocab - 1)[:, None]
    used = (ids >= 0) & (ids < vocab)
    ids = ids.clamp(0, vocab - 1)
    # the hard term
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    ce = lse - (1 - alpha) * logits.gather(1, target) - alpha * logits.mean(1, keepdim=True) + beta * lse * lse
    grad = (e / total).mul_((1 - mix) * (1 + 2 * beta * lse)).sub_((1 - mix) * alpha / vocab)
    grad.scatter_add_(1, target, torch.full_like(lse, -(1 - mix) * (1 - alpha)))
    # the soft term
    z = (s["teacher"].float() / tau).masked_fill(~used, -math.inf)
    z = z - z.amax(1, keepdim=True).clamp(min=-3e38)
    mass = torch.exp(z)
    has = used.any(1, keepdim=True)
    norm = torch.where(has, mass.sum(1, keepdim=True), 1.0)
    mass = mass / norm
    e = torch.exp((logits - top) / tau)
    total = e.sum(1, keepdim=True)
    log_p = (logits.gather(1, ids) - top) / tau - torch.log(total)
    log_t = z.masked_fill(~used, 0.0) - torch.log(norm)
    kd = tau * tau * (mass * (log_t - log_p)).sum(1, keepdim=True)
    grad.add_(torch.where(has, mix * tau * e / total, 0.0)).scatter_add_(1, ids, -mix * tau * mass)
    losses = torch.where(kept, torch.cat((ce, kd), 1), 0.0).t().contiguous()
    return losses, torch.where(kept, grad * inv_norm, 0.0)


_PLAIN = {"attention": _attention, "attention_backward": _attention_backward, "qk_norm_rope": _qk_norm_rope,
          "qk_norm_rope_backward": _qk_norm_rope_backward, "distill": _distill}


# --- the work a pass cannot do without ---


def work(case):
    if case["op"].startswith("attention"):
        hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]
        rows = sum(_lengths(case))
        pairs = 0
        for n in _lengths(case):
            i, w = np.arange(n, dtype=np.int64), case["window"] or n
            pairs += int(np.minimum(i + 1, w).sum())
            if not case["causal"]:
                pairs += int(np.minimum(n - 1 - i, w - 1).sum())
        if case["op"] == "attention":
            return {"bytes": 4 * rows * (2 * hq * dim + 2 * hkv * dim + hq), "flops": 4 * dim * hq * pairs}
        return {"bytes": 4 * rows * (4 * hq * dim + 4 * hkv * dim + hq), "flops": 10 * dim * hq * pairs}
    if case["op"].startswith("qk_norm_rope"):
        values = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * case["dim"]
        if case["op"] == "qk_norm_rope":
            return {"bytes": 8 * values, "flops": 7 * values}
        return {"bytes": 12 * values, "flops": 14 * values}
    values, top = case["rows"] * case["vocab"], case["rows"] * case["top"]
    return {"bytes": 8 * values + top * ((2 if case["half"] else 4) + (8 if case["wide_ids"] else 4))
            + 12 * case["rows"], "flops": 12 * values}


# --- the definitions in 64 bits ---


def exact(case, seed):
    state = prepare(case, seed)
    return _EXACT[case["op"]](case, state)


def _exact_heads(case, state):
    """For each sequence and query head: its rows, the shared head, and q, k, v of the two in 64 bits."""
    group = case["q_heads"] // case["kv_heads"]
    at = 0
    for n in _lengths(case):
        rows = slice(at, at + n)
        at += n
        i = torch.arange(n, device=DEVICE)
        hidden = torch.zeros(n, n, dtype=torch.bool, device=DEVICE)
        if case["causal"]:
            hidden |= i[None, :] > i[:, None]
        if case["window"]:
            hidden |= (i[None, :] - i[:, None]).abs() >= case["window"]
        for h in range(case["q_heads"]):
            q, k, v = (state[x][rows, y].double() for x, y in (("q", h), ("k", h // group), ("v", h // group)))
            scores = (q @ k.T) / math.sqrt(case["dim"])
            scores[hidden] = -math.inf
            yield rows, h, h // group, q, k, v, scores


def _exact_attention(case, state):
    tokens, heads, dim = state["q"].shape
    out = torch.zeros(tokens, heads, dim, dtype=torch.float64, device=DEVICE)
    lse = torch.full((heads, tokens), -math.inf, dtype=torch.float64, device=DEVICE)
    for rows, h, _, q, k, v, scores in _exact_heads(case, state):
        lse[h, rows] = torch.logsumexp(scores, 1)
        out[rows, h] = torch.softmax(scores, 1) @ v
    return out, lse


def _exact_attention_backward(case, state):
    dq, dk, dv = (torch.zeros(state[x].shape, dtype=torch.float64, device=DEVICE) for x in "qkv")
    for rows, h, hk, q, k, v, scores in _exact_heads(case, state):
        p = torch.exp(scores - state["lse"][h, rows].double()[:, None])
        do = state["dout"][rows, h].double()
        delta = (do * state["out"][rows, h].double()).sum(1)
        ds = p * (do @ v.T - delta[:, None]) / math.sqrt(case["dim"])
        dq[rows, h] = ds @ k
        dk[rows, hk] += ds.T @ q
        dv[rows, hk] += p.T @ do
    return dq, dk, dv


def _exact_turn(case, state):
    """The rotation of each token as complex factors of the pairs."""
    angle = torch.outer(state["positions"].double(), state["inv_freq"].double())
    return torch.polar(torch.ones_like(angle), angle)[:, None]


def _exact_rotate(case, x, turn):
    r = case["rotated"]
    y = x.clone()
    if case["interleaved"]:
        z = torch.complex(x[..., 0:r:2], x[..., 1:r:2]) * turn
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * turn
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    return y


def _exact_norm(x, w):
    return w * x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)


def _exact_qk_norm_rope(case, state):
    turn = _exact_turn(case, state)
    return tuple(_exact_rotate(case, _exact_norm(state[x].double(), state[x + "_weight"].double()), turn)
                 for x in ("q", "k"))


def _exact_qk_norm_rope_backward(case, state):
    turn = _exact_turn(case, state).conj()
    grads, weights = [], []
    for name in ("q", "k"):
        x = state[name].double().requires_grad_()
        w = state[name + "_weight"].double().requires_grad_()
        dn = _exact_rotate(case, state["d%s_out" % name].double(), turn)
        got = torch.autograd.grad(_exact_norm(x, w), (x, w), dn)
        grads.append(got[0])
        weights.append(got[1])
    return (*grads, *weights)


def _exact_distill(case, state):
    tau, mix, alpha, beta = case["temperature"], case["mix"], case["alpha"], case["beta"]
    rows, vocab = state["logits"].shape
    losses = torch.zeros(2, rows, dtype=torch.float64, device=DEVICE)
    grad = torch.empty(rows, vocab, dtype=torch.float64, device=DEVICE)
    for a in range(0, rows, 512):
        part = slice(a, min(a + 512, rows))
        l = state["logits"][part].double().requires_grad_()
        t, ids = state["targets"][part].long(), state["ids"][part].long()
        real = (t >= 0) & (t < vocab)
        lp = torch.log_softmax(l, 1)
        lse = torch.logsumexp(l, 1)
        ce = -(1 - alpha) * lp.gather(1, t.clamp(min=0)[:, None])[:, 0] - alpha * lp.mean(1) + beta * lse ** 2
        z = state["teacher"][part].double() / tau
        z[ids < 0] = -math.inf
        given = torch.log_softmax(z, 1)
        share = torch.where(ids < 0, 0.0, given.exp().nan_to_num(0.0))
        away = torch.where(ids < 0, 0.0, given - torch.log_softmax(l / tau, 1).gather(1, ids.clamp(min=0)))
        kd = tau ** 2 * (share * away.nan_to_num(0.0)).sum(1)
        losses[0, part] = torch.where(real, ce, 0.0).detach()
        losses[1, part] = torch.where(real, kd, 0.0).detach()
        total = (torch.where(real, (1 - mix) * ce + mix * kd, 0.0) * state["inv_norm"]).sum()
        grad[part] = torch.autograd.grad(total, l)[0]
    return losses, grad


_EXACT = {"attention": _exact_attention, "attention_backward": _exact_attention_backward,
          "qk_norm_rope": _exact_qk_norm_rope, "qk_norm_rope_backward": _exact_qk_norm_rope_backward,
          "distill": _exact_distill}
