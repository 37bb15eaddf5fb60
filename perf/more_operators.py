"""The operators between the linear layers of a transformer block that go beyond perf/operators.py, as they are
measured: attention whose scores are capped by a tanh, get a bias that falls with the distance, or are masked with a
prefix that is seen from everywhere; the norm of queries and keys with a rotation by positions of several axes; and the
norms behind and before a block, fused with the block's gate and the residual stream's update.  Each forward and
backward.

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
        # one short prompt through the 768-wide model's 12 heads, scores capped: launch latency counts
        {"name": "attention_capped_short", "op": "attention", "lengths": "93", "prefix": "", "tail": 0, "q_heads": 12,
         "kv_heads": 12, "dim": 64, "window": 0, "softcap": 30.0, "slopes": False},
        # prompts that are seen whole, each with its answer behind it, packed into one buffer; shared heads, a cap
        {"name": "attention_prefix_packed", "op": "attention", "lengths": "4096,1,613,2047,33,130,1999",
         "prefix": "1500,1,0,2047,20,64,700", "tail": 73, "q_heads": 16, "kv_heads": 4, "dim": 128, "window": 0,
         "softcap": 50.0, "slopes": False},
        # the 16 x 512-token batch of the 768-wide model, with a bias by distance whose slopes are learned
        {"name": "attention_backward_slopes16x512", "op": "attention_backward", "lengths": ",".join(["512"] * 16),
         "prefix": "", "tail": 0, "q_heads": 12, "kv_heads": 12, "dim": 64, "window": 0, "softcap": 0.0,
         "slopes": True},
        # one long document behind a prompt, shared heads, capped scores
        {"name": "attention_backward_capped_long", "op": "attention_backward", "lengths": "6143", "prefix": "1000",
         "tail": 0, "q_heads": 12, "kv_heads": 4, "dim": 64, "window": 0, "softcap": 30.0, "slopes": False},
        # an image of 23 x 22 patches for the 768-wide model: two axes
        {"name": "rope_axes_image", "op": "rope_axes", "tokens": 506, "axes": 2, "q_heads": 12, "kv_heads": 12,
         "dim": 64, "rotated": 64, "turns": False, "interleaved": False, "wide_positions": False},
        # 8 frames of 34 x 30 patches for a wider model with shared heads: time, height and width take turns
        {"name": "rope_axes_video", "op": "rope_axes", "tokens": 8160, "axes": 3, "q_heads": 24, "kv_heads": 8,
         "dim": 128, "rotated": 128, "turns": True, "interleaved": False, "wide_positions": True},
        # an odd number of tokens, part of each head rotated in neighbouring pairs
        {"name": "rope_axes_backward_odd", "op": "rope_axes_backward", "tokens": 1001, "axes": 3, "q_heads": 6,
         "kv_heads": 2, "dim": 96, "rotated": 48, "turns": False, "interleaved": True, "wide_positions": True},
        # a batch of 16 x 512 patches through the 768-wide model
        {"name": "rope_axes_backward_8192", "op": "rope_axes_backward", "tokens": 8192, "axes": 2, "q_heads": 12,
         "kv_heads": 12, "dim": 64, "rotated": 64, "turns": False, "interleaved": False, "wide_positions": False},
        # between two blocks of the 768-wide model at its training length, one learned gate
        {"name": "block_norm_512x768", "op": "block_norm", "lengths": "512", "tail": 0, "width": 768, "post": True,
         "gate": "shared", "residual_scale": 1.0, "block_scale": 1.0},
        # a packed batch of a wide model, gates of each sequence's condition, a scaled residual stream
        {"name": "block_norm_packed4096", "op": "block_norm", "lengths": "4096,1,613,2047,33,130,999", "tail": 73,
         "width": 4096, "post": True, "gate": "sequence", "residual_scale": 0.9, "block_scale": 0.5},
        # an odd width and number of tokens, no norm behind the block
        {"name": "block_norm_backward_odd", "op": "block_norm_backward", "lengths": "1001", "tail": 0, "width": 1150,
         "post": False, "gate": "shared", "residual_scale": 1.0, "block_scale": 1.0},
        # the 16 x 512-token batch of the 768-wide model, gates of each sequence's condition
        {"name": "block_norm_backward16x512", "op": "block_norm_backward", "lengths": ",".join(["512"] * 16),
         "tail": 0, "width": 768, "post": True, "gate": "sequence", "residual_scale": 1.0, "block_scale": 1.0},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _text(values):
    return ",".join(map(str, values))


def draw(rng):
    op = rng.choice(["attention", "attention_backward", "rope_axes", "rope_axes_backward", "block_norm",
                     "block_norm_backward"])
    if op.startswith("attention"):
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4])
        dim = rng.choice([32, 48, 64, 80, 96, 128])
        lengths = [_log_int(rng, 1, 4096) for _ in range(_log_int(rng, 1, 16))]
        # the padded scores of the plain form stay below those of the largest listed case
        while len(lengths) * heads * dim * max(lengths) ** 2 > 2 ** 34 or sum(lengths) > 8192:
            lengths[lengths.index(max(lengths))] = max(1, max(lengths) * 2 // 3)
        kind = rng.choice(["cap", "slopes", "prefix", "all"])
        prefix = [rng.choice([0, rng.randrange(n + 1)]) for n in lengths] if kind in ("prefix", "all") else []
        return {"op": op, "lengths": _text(lengths), "prefix": _text(prefix),
                "tail": rng.choice([0, rng.randrange(100)]), "q_heads": heads, "kv_heads": kv, "dim": dim,
                "window": rng.choice([0, 0, _log_int(rng, 1, 2000)]),
                "softcap": rng.choice([20.0, 30.0, 50.0]) if kind in ("cap", "all") else 0.0,
                "slopes": kind in ("slopes", "all")}
    if op.startswith("rope_axes"):
        kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([32, 64, 96, 128])
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "axes": rng.choice([2, 3, 4]),
                "q_heads": kv * rng.choice([1, 2, 3]), "kv_heads": kv, "dim": dim,
                "rotated": rng.choice([dim, dim // 2, 16]), "turns": rng.random() < 0.5,
                "interleaved": rng.random() < 0.5, "wide_positions": rng.random() < 0.5}
    width = rng.choice([_log_int(rng, 64, 8192), 4 * _log_int(rng, 16, 2048)])
    lengths = [_log_int(rng, 1, 4096) for _ in range(_log_int(rng, 1, 64))]
    while sum(lengths) * width > 2 ** 25 or sum(lengths) > 16384:
        lengths[lengths.index(max(lengths))] = max(1, max(lengths) * 2 // 3)
        if max(lengths) == 1 and len(lengths) * width > 2 ** 25:
            lengths = lengths[:max(1, 2 ** 25 // width)]
    return {"op": op, "lengths": _text(lengths), "tail": rng.choice([0, rng.randrange(100)]), "width": width,
            "post": rng.random() < 0.7, "gate": rng.choice(["none", "shared", "sequence"]),
            "residual_scale": rng.choice([1.0, round(rng.uniform(0.5, 2.0), 3)]),
            "block_scale": rng.choice([1.0, round(rng.uniform(0.1, 1.0), 3)])}


# --- what a user's program has in hand ---


def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


def _prefixes(case):
    return [int(x) for x in case["prefix"].split(",")] if case["prefix"] else [0] * len(_lengths(case))


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEVICE)

    if case["op"].startswith("attention"):
        return _prepare_attention(case, normal)
    if case["op"].startswith("rope_axes"):
        return _prepare_rope(case, normal, g)
    return _prepare_block(case, normal)


def _cu(lengths):
    return torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32, device=DEVICE)


def _prepare_attention(case, normal):
    lengths = _lengths(case)
    tokens = sum(lengths) + case["tail"]
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    # queries, keys and values as one projection writes them; scores of several units, so that a cap bends some
    qkv = normal(tokens, (hq + 2 * hkv) * dim)
    qkv[:, :hq * dim] *= 4.0
    q, k, v = qkv.split([hq * dim, hkv * dim, hkv * dim], dim=1)
    state = {"case": case, "q": q.view(tokens, hq, dim), "k": k.view(tokens, hkv, dim), "v": v.view(tokens, hkv, dim),
             "cu_seqlens": _cu(lengths), "longest": max(lengths), "slopes": None, "prefix_lens": None}
    if case["slopes"]:
        state["slopes"] = torch.exp2(-8.0 * (1.0 + torch.arange(hq, device=DEVICE, dtype=torch.float32)) / hq)
    if case["prefix"]:
        state["prefix_lens"] = torch.tensor(_prefixes(case), dtype=torch.int32, device=DEVICE)
    if case["op"] == "attention_backward":
        state["out"], state["lse"] = _attention(state)
        state["dout"] = normal(tokens, hq, dim)
    return state


def _prepare_rope(case, normal, g):
    tokens, hq, hkv, dim = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    axes, pairs = case["axes"], case["rotated"] // 2
    qkv = normal(tokens, (hq + 2 * hkv) * dim)
    # the place of each token on a grid whose last axis runs fastest, every axis from an offset of its own
    side = max(1, round(tokens ** (1.0 / axes)))
    token = torch.arange(tokens, device=DEVICE, dtype=torch.int64)
    places = [token // side ** (axes - 1)] + [token // side ** (axes - 1 - a) % side for a in range(1, axes)]
    first = torch.randint(1000, (axes, 1), generator=g, device=DEVICE)
    positions = torch.stack(places) + first
    pair = torch.arange(pairs, device=DEVICE)
    axis = pair % axes if case["turns"] else pair * axes // max(1, pairs)
    state = {"case": case, "q": qkv[:, :hq * dim].view(tokens, hq, dim),
             "k": qkv[:, hq * dim:(hq + hkv) * dim].view(tokens, hkv, dim),
             "q_weight": 1.0 + 0.1 * normal(dim), "k_weight": 1.0 + 0.1 * normal(dim),
             "positions": positions if case["wide_positions"] else positions.int(), "pair_axis": axis.int(),
             "inv_freq": torch.tensor(10000.0 ** (-np.arange(pairs) / pairs), dtype=torch.float32, device=DEVICE)}
    if case["op"] == "rope_axes_backward":
        state["dq_out"], state["dk_out"] = normal(tokens, hq, dim), normal(tokens, hkv, dim)
    return state


def _prepare_block(case, normal):
    lengths, width = _lengths(case), case["width"]
    tokens = sum(lengths) + case["tail"]
    state = {"case": case, "y": normal(tokens, width), "pre_weight": 1.0 + 0.1 * normal(width),
             "post_weight": 1.0 + 0.1 * normal(width) if case["post"] else None, "gate": None, "cu_seqlens": None}
    if case["gate"] == "shared":
        state["gate"] = 0.5 + 0.2 * normal(width)
    if case["gate"] == "sequence":
        state["gate"] = 0.5 + 0.2 * normal(len(lengths), width)
    if case["gate"] == "sequence" or case["tail"] or len(lengths) > 1:
        state["cu_seqlens"] = _cu(lengths)
    if case["op"] == "block_norm":
        state["x"] = 2.0 * normal(tokens, width)
    else:
        state["x_out"] = 2.0 * normal(tokens, width)
        state["dx_out"], state["dh"] = normal(tokens, width), normal(tokens, width)
    return state


# --- one pass ---


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_attention(s):
    from tiled_dense_gemm_matmul_amd import binding
    c = s["case"]
    return binding.attention(s["q"], s["k"], s["v"], cu_seqlens=s["cu_seqlens"], causal=True, window=c["window"],
                             softcap=c["softcap"], slopes=s["slopes"], prefix_lens=s["prefix_lens"])


def _own_attention_backward(s):
    from tiled_dense_gemm_matmul_amd import binding
    c = s["case"]
    dslopes = torch.empty_like(s["slopes"]) if c["slopes"] else None
    return binding.attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"],
                                      cu_seqlens=s["cu_seqlens"], causal=True, window=c["window"],
                                      softcap=c["softcap"], slopes=s["slopes"], prefix_lens=s["prefix_lens"],
                                      dslopes=dslopes)


def _own_rope_axes(s):
    from tiled_dense_gemm_matmul_amd import binding
    return binding.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"], eps=1e-6,
                                interleaved=s["case"]["interleaved"], pair_axis=s["pair_axis"])


def _own_rope_axes_backward(s):
    from tiled_dense_gemm_matmul_amd import binding
    return binding.qk_norm_rope_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["q_weight"], s["k_weight"],
                                         s["positions"], s["inv_freq"], eps=1e-6,
                                         interleaved=s["case"]["interleaved"], pair_axis=s["pair_axis"])


def _own_block_norm(s):
    from tiled_dense_gemm_matmul_amd import binding
    c = s["case"]
    return binding.block_norm(s["x"], s["y"], s["pre_weight"], post_weight=s["post_weight"], gate=s["gate"],
                              residual_scale=c["residual_scale"], block_scale=c["block_scale"],
                              cu_seqlens=s["cu_seqlens"], eps=1e-6)


def _own_block_norm_backward(s):
    from tiled_dense_gemm_matmul_amd import binding
    c = s["case"]
    grads = binding.block_norm_backward(s["dx_out"], s["dh"], s["x_out"], s["y"], s["pre_weight"],
                                        post_weight=s["post_weight"], gate=s["gate"],
                                        residual_scale=c["residual_scale"], block_scale=c["block_scale"],
                                        cu_seqlens=s["cu_seqlens"], eps=1e-6)
    return [g for g in grads if g is not None]  # no gradient of a weight or gate that is not there


_OWN = {"attention": _own_attention, "attention_backward": _own_attention_backward, "rope_axes": _own_rope_axes,
        "rope_axes_backward": _own_rope_axes_backward, "block_norm": _own_block_norm,
        "block_norm_backward": _own_block_norm_backward}


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
        self.distance = gap.abs().float()
        sees = (gap >= 0)[None]
        if s["prefix_lens"] is not None:
            sees = sees | (pos[None, None, :] < s["prefix_lens"].long()[:, None, None])
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


def _scores(s, p, q, k, groups):
    """The final scores [sequences, kv_heads, groups, rows, keys], and the derivative of the cap (None without)."""
    cap, bent = s["case"]["softcap"], None
    b, hkv, rows, dim = q.shape
    t = torch.matmul(q, k.transpose(2, 3)).mul_(dim ** -0.5).view(b, hkv, groups, rows // groups, k.shape[2])
    if cap:
        t = t.div_(cap).tanh_()
        bent = 1.0 - t * t
        t = t.mul_(cap)
    if s["slopes"] is not None:
        t = t.sub_(s["slopes"].view(hkv, groups, 1, 1) * p.distance)
    return t.masked_fill_(~p.mask, -math.inf), bent


def _attention(s):
    q, k, v = s["q"], s["k"], s["v"]
    heads, groups, p = q.shape[1], q.shape[1] // k.shape[1], _Packing(s)
    scores, _ = _scores(s, p, p.pad(q, groups), p.pad(k), groups)
    top = scores.amax(-1, keepdim=True).clamp_(min=-3e38)
    probs = torch.exp(scores.sub_(top))
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
    scores, bent = _scores(s, p, qp, kp, groups)
    probs = torch.exp(scores.flatten(2, 3) - lse)
    probs = torch.where(p.mask.expand(scores.shape).flatten(2, 3), probs, 0.0)
    ds = probs * (torch.matmul(dp, vp.transpose(2, 3)) - delta)
    grads = []
    if s["slopes"] is not None:
        away = ds.view(scores.shape) * p.distance
        grads.append(-away.sum((0, 3, 4), dtype=torch.float64).float().flatten())  # a long sum
    if bent is not None:
        ds = ds * bent.flatten(2, 3)
    dq = torch.matmul(ds, kp) * scale
    dk = torch.matmul(ds.transpose(2, 3), qp) * scale
    dv = torch.matmul(probs.transpose(2, 3), dp)
    return (p.unpad(dq, heads), p.unpad(dk, kv_heads), p.unpad(dv, kv_heads), *grads)


def _cos_sin(s):
    # far positions need 64 bits
    angle = s["positions"][s["pair_axis"].long()].t().double() * s["inv_freq"].double()[None, :]
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


def _rope_axes(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    result = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        a, b, rest = _halves(y, c["rotated"], c["interleaved"])
        result.append(_join(a * cos - b * sin, b * cos + a * sin, rest, c["interleaved"]))
    return result[0], result[1]


def _norm_backward(g, x, r):
    """The gradient of x r from g, r the reciprocal root mean square of x."""
    n = x * r
    return r * (g - n * (g * n).mean(-1, keepdim=True))


def _rope_axes_backward(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    grads, weights = [], []
    for dy, x, w in ((s["dq_out"], s["q"], s["q_weight"]), (s["dk_out"], s["k"], s["k_weight"])):
        a, b, rest = _halves(dy, c["rotated"], c["interleaved"])
        dn = _join(a * cos + b * sin, b * cos - a * sin, rest, c["interleaved"])
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        grads.append(_norm_backward(dn * w, x, r))
        weights.append((dn * x * r).sum((0, 1), dtype=torch.float64).float())  # a long sum
    return grads[0], grads[1], weights[0], weights[1]


def _rows(s, tokens):
    """The sequence of each row, and which rows belong to one."""
    row = torch.arange(tokens, device=DEVICE)
    if s["cu_seqlens"] is None:
        return torch.zeros_like(row), torch.ones_like(row, dtype=torch.bool)[:, None]
    cu = s["cu_seqlens"].long()
    seq = torch.searchsorted(cu, row, right=True) - 1
    return seq.clamp(0, len(cu) - 2), ((row >= cu[0]) & (row < cu[-1]))[:, None]


def _gates(s, seq):
    gate = s["gate"]
    if gate is None:
        return 1.0
    return gate if gate.dim() == 1 else gate[seq]


def _block_norm(s):
    c, x, y = s["case"], s["x"], s["y"]
    seq, used = _rows(s, x.shape[0])
    if c["post"]:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * s["post_weight"]
    out = c["residual_scale"] * x + c["block_scale"] * _gates(s, seq) * y
    out = torch.where(used, out, 0.0)
    h = out * torch.rsqrt((out * out).mean(-1, keepdim=True) + 1e-6) * s["pre_weight"]
    return out, h


def _block_norm_backward(s):
    c, out, y, dh = s["case"], s["x_out"], s["y"], s["dh"]
    seq, used = _rows(s, out.shape[0])
    r = torch.rsqrt((out * out).mean(-1, keepdim=True) + 1e-6)
    dx_out = torch.where(used, s["dx_out"] + _norm_backward(dh * s["pre_weight"], out, r), 0.0)
    grads = [c["residual_scale"] * dx_out]
    weights = [torch.where(used, dh * out * r, 0.0).sum(0, dtype=torch.float64).float()]  # long sums
    u = c["block_scale"] * dx_out
    n = y
    dn = u * _gates(s, seq)
    if c["post"]:
        ry = torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)
        n = y * ry
        weights.append((dn * n).sum(0, dtype=torch.float64).float())
        grads.append(_norm_backward(dn * s["post_weight"], y, ry))
        n = n * s["post_weight"]
    else:
        grads.append(dn)
    if c["gate"] == "shared":
        weights.append((u * n).sum(0, dtype=torch.float64).float())
    if c["gate"] == "sequence":
        member = (seq == torch.arange(len(s["gate"]), device=DEVICE)[:, None]).double()
        weights.append((member @ (u * n).double()).float())
    return grads + weights


_PLAIN = {"attention": _attention, "attention_backward": _attention_backward, "rope_axes": _rope_axes,
          "rope_axes_backward": _rope_axes_backward, "block_norm": _block_norm,
          "block_norm_backward": _block_norm_backward}


# --- the work a pass cannot do without ---


def work(case):
    if case["op"].startswith("attention"):
        hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]
        rows = sum(_lengths(case))
        pairs = 0
        for n, first in zip(_lengths(case), _prefixes(case)):
            i, w = np.arange(n, dtype=np.int64), case["window"] or n
            last = np.minimum(np.maximum(i + 1, min(first, n)), i + w)
            pairs += int((last - np.maximum(i - w + 1, 0)).sum())
        if case["op"] == "attention":
            return {"bytes": 4 * rows * (2 * hq * dim + 2 * hkv * dim + hq), "flops": 4 * dim * hq * pairs}
        return {"bytes": 4 * rows * (4 * hq * dim + 4 * hkv * dim + hq), "flops": 10 * dim * hq * pairs}
    if case["op"].startswith("rope_axes"):
        values = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * case["dim"]
        places = case["tokens"] * case["axes"] * (8 if case["wide_positions"] else 4)
        if case["op"] == "rope_axes":
            return {"bytes": 8 * values + places, "flops": 7 * values}
        return {"bytes": 12 * values + places, "flops": 14 * values}
    values = sum(_lengths(case)) * case["width"]
    gates = {"none": 0, "shared": 1, "sequence": len(_lengths(case))}[case["gate"]] * case["width"]
    if case["op"] == "block_norm":
        return {"bytes": 16 * values + 4 * gates, "flops": 12 * values}
    return {"bytes": 24 * values + 8 * gates, "flops": 30 * values}


# --- the definitions in 64 bits ---


def exact(case, seed):
    state = prepare(case, seed)
    return _EXACT[case["op"]](case, state)


def _exact_heads(case, state):
    """For each sequence and query head: its rows, the shared head, q, k, v of the two in 64 bits, the final scores,
    the derivative of the cap and the distances."""
    group, cap = case["q_heads"] // case["kv_heads"], case["softcap"]
    at = 0
    for n, first in zip(_lengths(case), _prefixes(case)):
        rows = slice(at, at + n)
        at += n
        i = torch.arange(n, device=DEVICE)
        away = (i[None, :] - i[:, None]).abs()
        hidden = (i[None, :] > i[:, None]) & (i[None, :] >= first)
        if case["window"]:
            hidden |= away >= case["window"]
        away = away.double()
        for h in range(case["q_heads"]):
            q, k, v = (state[x][rows, y].double() for x, y in (("q", h), ("k", h // group), ("v", h // group)))
            scores = (q @ k.T) / math.sqrt(case["dim"])
            bent = 1.0
            if cap:
                bent = 1.0 / torch.cosh(scores / cap).square()
                scores = cap * torch.tanh(scores / cap)
            if case["slopes"]:
                scores = scores - state["slopes"][h].double() * away
            scores[hidden] = -math.inf
            yield rows, h, h // group, q, k, v, scores, bent, away


def _exact_attention(case, state):
    tokens, heads, dim = state["q"].shape
    out = torch.zeros(tokens, heads, dim, dtype=torch.float64, device=DEVICE)
    lse = torch.full((heads, tokens), -math.inf, dtype=torch.float64, device=DEVICE)
    for rows, h, _, _, _, v, scores, _, _ in _exact_heads(case, state):
        lse[h, rows] = torch.logsumexp(scores, 1)
        out[rows, h] = torch.softmax(scores, 1) @ v
    return out, lse


def _exact_attention_backward(case, state):
    dq, dk, dv = (torch.zeros(state[x].shape, dtype=torch.float64, device=DEVICE) for x in "qkv")
    dslopes = torch.zeros(case["q_heads"], dtype=torch.float64, device=DEVICE)
    for rows, h, hk, q, k, v, scores, bent, away in _exact_heads(case, state):
        p = torch.exp(scores - state["lse"][h, rows].double()[:, None])
        do = state["dout"][rows, h].double()
        delta = (do * state["out"][rows, h].double()).sum(1)
        ds = p * (do @ v.T - delta[:, None])
        dslopes[h] -= (ds * away).sum()
        ds = ds * bent / math.sqrt(case["dim"])
        dq[rows, h] = ds @ k
        dk[rows, hk] += ds.T @ q
        dv[rows, hk] += p.T @ do
    return (dq, dk, dv, dslopes) if case["slopes"] else (dq, dk, dv)


def _exact_turn(state):
    """The rotation of each token as complex factors of the pairs."""
    places = state["positions"].double().index_select(0, state["pair_axis"].long())
    angle = (places * state["inv_freq"].double()[:, None]).T
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


def _exact_rope_axes(case, state):
    turn = _exact_turn(state)
    return tuple(_exact_rotate(case, _exact_norm(state[x].double(), state[x + "_weight"].double()), turn)
                 for x in ("q", "k"))


def _exact_rope_axes_backward(case, state):
    turn = _exact_turn(state).conj()
    grads, weights = [], []
    for name in ("q", "k"):
        x = state[name].double().requires_grad_()
        w = state[name + "_weight"].double().requires_grad_()
        dn = _exact_rotate(case, state["d%s_out" % name].double(), turn)
        got = torch.autograd.grad(_exact_norm(x, w), (x, w), dn)
        grads.append(got[0])
        weights.append(got[1])
    return (*grads, *weights)


def _exact_branch(case, y, weight, gate):
    """What a block adds to the rows of one sequence."""
    n = _exact_norm(y, weight) if case["post"] else y
    return case["block_scale"] * (n if gate is None else gate * n)


def _exact_gate(case, gate, sequence):
    return gate[sequence] if case["gate"] == "sequence" else gate


def _doubles(*tensors):
    return [None if t is None else t.double() for t in tensors]


def _exact_block_norm(case, state):
    x, y, pre, post, gate = _doubles(*(state[n] for n in ("x", "y", "pre_weight", "post_weight", "gate")))
    out, h, at = torch.zeros_like(x), torch.zeros_like(x), 0
    for b, n in enumerate(_lengths(case)):
        rows = slice(at, at + n)
        at += n
        out[rows] = case["residual_scale"] * x[rows] + _exact_branch(case, y[rows], post, _exact_gate(case, gate, b))
        h[rows] = _exact_norm(out[rows], pre)
    return out, h


def _exact_block_norm_backward(case, state):
    y, pre, post, gate = _doubles(*(state[n] for n in ("y", "pre_weight", "post_weight", "gate")))
    out, dx_out, dh = _doubles(*(state[n] for n in ("x_out", "dx_out", "dh")))
    dx, dy, at = torch.zeros_like(out), torch.zeros_like(out), 0
    leaves = [w.requires_grad_() for w in (pre, post, gate) if w is not None]
    sums = [torch.zeros_like(w) for w in leaves]
    for b, n in enumerate(_lengths(case)):
        rows = slice(at, at + n)
        at += n
        o, yb = out[rows].clone().requires_grad_(), y[rows].clone().requires_grad_()
        through, dpre = torch.autograd.grad(_exact_norm(o, pre), (o, pre), dh[rows])
        dt = dx_out[rows] + through
        dx[rows] = case["residual_scale"] * dt
        got = torch.autograd.grad(_exact_branch(case, yb, post, _exact_gate(case, gate, b)), [yb, *leaves[1:]], dt)
        dy[rows] = got[0]
        for total, part in zip(sums, (dpre, *got[1:])):
            total += part
    return [dx, dy, *sums]


_EXACT = {"attention": _exact_attention, "attention_backward": _exact_attention_backward,
          "rope_axes": _exact_rope_axes, "rope_axes_backward": _exact_rope_axes_backward,
          "block_norm": _exact_block_norm, "block_norm_backward": _exact_block_norm_backward}
