"""attention and attention_backward on the GPU against the oracle
(oracle/attention.py): every head width of the kernels and widths between
them, shared heads, causal and sliding-window masks, packed sequences of one
token, of none, and ending anywhere in a tile, strided views, rows of no
sequence, poisoned neighbours, offsets past 32 bits, other streams and graph
replays.  The bounds are the oracle's, counted per element."""
import numpy as np
import pytest

from oracle import attention as OA

from _gpu import device, say, to_dev

pytestmark = pytest.mark.gpu

SENTINEL = -777.0


def cu_of(lengths, first=0):
    return np.cumsum([first] + list(lengths)).astype(np.int32)


class Case:
    """Device tensors of an attention call: q, k, v as views in `layout`,
    everything around them NaN, rows of no sequence NaN as well."""

    def __init__(self, seed, lengths, first=0, tail=0, hq=2, hk=1, d=64, layout="qkv", causal=True, window=0,
                 scale=None, gain=1.0):
        import torch
        r = np.random.default_rng(seed)
        self.T = T = first + sum(lengths) + tail
        self.kw = {"causal": causal, "window": window, "scale": scale}
        self.cu = None if lengths == [T] else cu_of(lengths, first)
        self.shapes = ((T, hq, d), (T, hk, d), (T, hk, d))
        self.host = [(r.standard_normal(s) * gain).astype(np.float32) for s in self.shapes]
        self.g = r.standard_normal(self.shapes[0]).astype(np.float32)
        self.used = np.zeros(T, bool)
        for a, b in OA.sequences(self.cu, T):
            self.used[a:b] = True
        self.layout = layout
        self.q, self.k, self.v = self.fill(self.views(float("nan")), self.host)
        self.dcu = None if self.cu is None else to_dev(self.cu)
        (self.dout,) = self.fill([torch.full(self.shapes[0], float("nan"), device=device())], [self.g])

    def views(self, value):
        """Three tensors of the q, k, v shapes in this case's layout, filled with `value`."""
        import torch
        T = self.T
        if self.layout == "qkv":      # one projection's columns, 4 unused ones behind
            w = [s[1] * s[2] for s in self.shapes]
            buf = torch.full((T, sum(w) + 4), value, device=device())
            self.buffer = buf
            at = np.cumsum([0] + w)
            return [buf[:, at[i]:at[i + 1]].unflatten(1, self.shapes[i][1:]) for i in range(3)]
        if self.layout == "heads":    # [heads, tokens, head_dim], 8 unused rows a head
            return [torch.full((s[1], T + 8, s[2]), value, device=device())[:, :T].transpose(0, 1)
                    for s in self.shapes]
        return [torch.full(s, value, device=device()) for s in self.shapes]

    def fill(self, views, arrays):
        for t, a in zip(views, arrays):
            rows = to_dev(np.flatnonzero(self.used))
            t[rows] = to_dev(a[self.used])
        return views

    def clean(self, a):
        return np.where(self.used[:, None, None], a, 0.0)

    def oracle_args(self):
        kw = dict(self.kw)
        return [self.clean(x) for x in self.host], {"cu": self.cu, **kw}


def call(c, **kw):
    from tiled_dense_gemm_matmul_amd import binding
    return binding.attention(c.q, c.k, c.v, cu_seqlens=c.dcu, **c.kw, **kw)


def call_backward(c, out, lse, **kw):
    from tiled_dense_gemm_matmul_amd import binding
    return binding.attention_backward(c.dout, c.q, c.k, c.v, out, lse, cu_seqlens=c.dcu, **c.kw, **kw)


def check(c, label):
    import torch
    out, lse = call(c)
    torch.cuda.synchronize()
    args, kw = c.oracle_args()
    ro, rl, eo, el = OA.attention(*args, **kw)
    for name, y, ref, err in (("out", out, ro, eo), ("lse", lse, rl, el)):
        res = OA.compare(y.cpu().numpy(), ref, err)
        say(f"  {label} {name}: max err/bound {res['max_ratio']:.3g}, fails {res['fails']} of {res['n']}")
        assert res["fails"] == 0, (label, name, res)
    got = call_backward(c, out, lse)
    torch.cuda.synchronize()
    # from the out and lse that the call was given
    want = OA.attention_backward(c.clean(c.g), *args, out.cpu().numpy(), lse.cpu().numpy(), **kw)
    for name, y, ref, err in zip(("dq", "dk", "dv"), got, want[:3], want[3:]):
        res = OA.compare(y.cpu().numpy(), ref, err)
        say(f"  {label} {name}: max err/bound {res['max_ratio']:.3g}, fails {res['fails']} of {res['n']}")
        assert res["fails"] == 0, (label, name, res)


@pytest.mark.parametrize("d", [4, 12, 20, 32, 36, 48, 64, 72, 80, 96, 100, 128])
def test_head_widths(d):
    say(f"attention head_dim {d}")
    check(Case(d, [70, 33], hq=2, hk=1, d=d), f"D={d}")


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 37), (False, 1), (False, 37)])
def test_masks_on_many_rows(d, causal, window):
    """Enough heads and rows that a workgroup's waves hold their own rows."""
    say(f"attention D={d} causal={causal} window={window}")
    check(Case(d + window, [300, 1, 0, 131, 80], first=3, tail=7, hq=96, hk=96, d=d, causal=causal, window=window,
               layout="dense"), f"D={d} {causal} {window}")


# one problem for each way the kernels deal out rows and keys: few rows, many
# rows, shared heads, and many short sequences, with widths that fill the
# kernels' and that do not
PLANS = {"few": dict(lengths=[900], hq=8, hk=8), "many": dict(lengths=[520], tail=3, hq=64, hk=64),
         "shared": dict(lengths=[300, 33], hq=32, hk=2),
         "short": dict(lengths=[200, 1, 0, 130, 120, 77], first=2, tail=9, hq=128, hk=128)}


@pytest.mark.parametrize("d", [20, 32, 48, 64, 80, 96, 100, 128])
@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 70)])
def test_plans(plan, d, causal, window):
    say(f"attention {plan} D={d} causal={causal} window={window}")
    check(Case(d, d=d, causal=causal, window=window, **PLANS[plan]), f"{plan} D={d}")


@pytest.mark.parametrize("lengths", [[1], [2], [15], [16], [17], [63], [64], [65], [1] * 40, [0, 5, 0, 0, 3, 0],
                                     [127, 129], [513], list(range(1, 24))])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths(lengths, causal):
    say(f"attention lengths {lengths} causal={causal}")
    check(Case(len(lengths), lengths, hq=3, hk=3, d=32, causal=causal), str(lengths)[:30])


@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 1), (6, 2), (5, 5), (16, 2), (200, 50)])
@pytest.mark.parametrize("layout", ["qkv", "heads", "dense"])
def test_shared_heads_and_layouts(hq, hk, layout):
    say(f"attention heads {hq}/{hk} {layout}")
    check(Case(hq, [200, 57], first=1, tail=5, hq=hq, hk=hk, d=64, layout=layout, window=90), f"{hq}/{hk} {layout}")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,longest", [(2, 9), (64, 40)])
def test_many_sequences(causal, heads, longest):
    """More sequences than one look of 64 finds, some empty, some of several tiles."""
    r = np.random.default_rng(3)
    lengths = [int(x) for x in r.integers(0, longest, 300)]
    lengths[70], lengths[200] = 150, 70
    check(Case(4, lengths, tail=3, hq=heads, hk=heads, d=32, causal=causal), "300 sequences")


@pytest.mark.parametrize("number", [512, 513, 4095, 4097, 9000])
@pytest.mark.parametrize("causal", [True, False])
def test_thousands_of_sequences(number, causal):
    """On both sides of the number from which a tile's sequence is searched
    for, and of those at which that search takes another look: sequences of no
    rows to a few, runs of empty ones, and some of several tiles."""
    r = np.random.default_rng(number)
    lengths = r.choice(4, number)
    lengths[100:300] = 0
    lengths[[0, 63, 64, 301, number - 2]] = 50, 70, 33, 17, 40
    lengths[number // 2] = 150
    check(Case(number, [int(n) for n in lengths], first=5, tail=3, hq=2, hk=1, d=32, causal=causal), f"{number} sequences")


@pytest.mark.parametrize("heads,longest", [(48, 40), (48, 200), (3, 400)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 30)])
def test_hundreds_of_sequences_on_longer_tiles(heads, longest, causal, window):
    """The same with tiles of 32 and 128 rows."""
    r = np.random.default_rng(longest)
    lengths = [int(n) for n in r.integers(0, longest, 560) * (r.random(560) < (0.9 if longest == 40 else 0.1))]
    check(Case(longest, lengths, first=2, tail=70, hq=heads, hk=heads, d=32, causal=causal, window=window),
          f"560 sequences, {heads} heads")


@pytest.mark.parametrize("front", [True, False])
def test_most_sequences(front):
    """As many entries in cu_seqlens as a call takes, all but a few of them
    empty, in front of the others or behind them: the bits of the few alone."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    g = torch.Generator(device=device())
    g.manual_seed(6)
    few = cu_of([300, 1, 40, 500, 97], first=10)
    T = int(few[-1]) + 12
    q, k, v, do = (torch.randn((T, 1, 32), generator=g, device=device()) for _ in range(4))
    n = (1 << 24) - len(few)
    cu = torch.full((n,), int(few[0] if front else few[-1]), dtype=torch.int32, device=device())
    cu, few = torch.cat((cu, to_dev(few)) if front else (to_dev(few), cu)), to_dev(few)
    assert cu.shape[0] - 1 == (1 << 24) - 1
    out, lse = binding.attention(q, k, v, cu_seqlens=cu)
    want = binding.attention(q, k, v, cu_seqlens=few)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    grads = binding.attention_backward(do, q, k, v, out, lse, cu_seqlens=cu)
    want = binding.attention_backward(do, q, k, v, out, lse, cu_seqlens=few)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))


@pytest.mark.parametrize("gain,scale", [(6.0, None), (1.0, 2.5), (0.01, 1e-4)])
def test_scales(gain, scale):
    """Scores from nearly equal to ones whose exponentials underflow."""
    check(Case(9, [150], hq=2, hk=2, d=64, gain=gain, scale=scale), f"gain {gain} scale {scale}")


@pytest.mark.parametrize("tokens,heads", [(40, 1), (128, 512)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_near_the_largest(sign, tokens, heads):
    """Scores up to 1.4 2^29, 2^20 and more apart: each row takes one key's
    value.  That value is multiplied by a probability, divided by the same
    one (a reciprocal and a product) and rounded each time, so it is off by
    less than 2^-21 of itself.  lse is the largest score through the product
    with scale log2(e) and back with ln 2, four roundings and two constants'
    of 2^-24, and the logarithm of a sum of up to 2^63, another 2^-24."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    dev = device()
    r = np.random.default_rng(12)
    q = torch.zeros((tokens, heads, 32), device=dev)
    k, v = torch.zeros_like(q), to_dev(r.standard_normal((tokens, heads, 32)).astype(np.float32))
    steps = (1.0 + torch.arange(tokens, device=dev) / (4.0 * tokens)) * 1.1
    q[:, :, 3] = 2.0 ** 14
    k[:, :, 3] = (sign * 2.0 ** 15 * steps)[:, None]
    out, lse = binding.attention(q, k, v, causal=False, scale=1.0)
    torch.cuda.synchronize()
    best = tokens - 1 if sign > 0 else 0
    score = float(q[0, 0, 3].double() * k[best, 0, 3].double())
    err = (out.double() - v[best].double()).abs()
    assert bool((err <= 2.0 ** -21 * v[best].double().abs()).all())
    assert bool(((lse.double() - score).abs() <= 2.0 ** -21 * abs(score)).all())


# the ways the backward pass deals out rows: few (delta formed within), many, and many short sequences' worth
LARGE = {"few": (40, 1), "many": (1024, 32), "short": (128, 512)}


@pytest.mark.parametrize("shape", LARGE)
@pytest.mark.parametrize("d,scale", [(20, 0.37), (32, None), (64, None), (128, None)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_gradients_of_large_scores(shape, d, scale, sign):
    """Scores from 2^12 to 2^30 in magnitude, of rows that see one key and of
    rows that see all of them, one 2^-12 of the score or more above the rest
    (exp of -256 is below every fp32 number).  The one key's probability is 1 whatever its score:
    lse is the score in fp32 (q holds one power of two, so q.k is exact and
    the product with scale its only rounding) and dv of a row that only itself
    sees is its dout, both to the bit; dv of the best key is the sum of all
    rows' dout and of the others zero.  ds is dout.v - dout.out, two sums of d
    products each off by (d + 1) u, with an out that is off by 2^-21; dq and
    dk are its products with k and q."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    T, heads = LARGE[shape]
    u, factor = 2.0 ** -24, np.float32(d ** -0.5 if scale is None else scale)
    g = torch.Generator(device=device())
    g.manual_seed(d)
    v, do = (torch.randn((T, heads, d), generator=g, device=device()) for _ in range(2))
    size = (do * v).abs().double().sum(2)
    for power in (12, 20, 24, 29):
        q, k = torch.zeros_like(v), torch.zeros_like(v)
        q[:, :, 3] = 2.0 ** (power // 2)
        key = sign * 2.0 ** (power - power // 2) / float(factor)
        # one visible key, of any score
        k[:, :, 3] = key * (1.0 + 0.9 * torch.rand((T, heads), generator=g, device=device()))
        out, lse = binding.attention(q, k, v, window=1, scale=scale)
        dq, dk, dv = binding.attention_backward(do, q, k, v, out, lse, window=1, scale=scale)
        score = (q[:, :, 3] * k[:, :, 3]).cpu().numpy() * factor
        assert np.array_equal(lse.t().cpu().numpy(), score), (power, "lse")
        assert torch.equal(dv, do), (power, "dv")
        e = (2 * (d + 2) * u + 2.0 ** -21) * size * float(factor) * (1 + 8 * u)
        assert bool((dq[:, :, 3].double().abs() <= e * k[:, :, 3].double().abs()).all()), (power, "dq")
        assert bool((dk[:, :, 3].double().abs() <= e * q[:, :, 3].double().abs()).all()), (power, "dk")
        if power < 20:
            continue
        # all keys, one of them far above the rest
        steps = 1.0 + torch.arange(T, device=device()) / (4.0 * T)
        k[:, :, 3] = (key * steps * 1.1)[:, None]
        best = T - 1 if sign > 0 else 0
        out, lse = binding.attention(q, k, v, causal=False, scale=scale)
        dq, dk, dv = binding.attention_backward(do, q, k, v, out, lse, causal=False, scale=scale)
        score = (q[0, 0, 3] * k[best, 0, 3]).cpu().numpy() * factor
        assert bool((lse == float(score)).all()), (power, "lse of many")
        total, most = do.double().sum(0), do.double().abs().sum(0)
        assert bool(((dv[best].double() - total).abs() <= (T + 2) * u * most).all()), (power, "dv of many")
        dv[best], dk_best = 0.0, dk[best].clone()
        dk[best] = 0.0
        assert not dv.any() and not dk.any(), power
        e = (2 * (d + 2) * u + 2.0 ** -21) * (do * v[best]).abs().double().sum(2) * float(factor) * (1 + (T + 8) * u)
        assert bool((dq[:, :, 3].double().abs() <= e * k[best, 0, 3].double().abs()).all()), (power, "dq of many")
        assert bool((dk_best[:, 3].double().abs() <= e.sum(0) * 2.0 ** (power // 2)).all()), (power, "dk of many")


def test_empty():
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    dev = device()
    q = torch.empty((0, 2, 32), device=dev)
    out, lse = binding.attention(q, q, q)
    assert out.shape == (0, 2, 32) and lse.shape == (2, 0)
    assert [x.shape for x in binding.attention_backward(q, q, q, q, out, lse)] == [(0, 2, 32)] * 3
    # no sequence at all: every row is outside
    q = torch.full((37, 2, 32), float("nan"), device=dev)
    cu = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = binding.attention(q, q, q, cu_seqlens=cu)
    grads = binding.attention_backward(q, q, q, q, q, lse, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert not out.any() and bool((lse == -float("inf")).all()) and not any(bool(x.any()) for x in grads)


def test_bounds_of_sequences_are_clamped():
    """Entries outside [0, tokens] read as the nearest bound."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    c = Case(5, [50], hq=2, hk=1, d=32, layout="dense")
    far = torch.tensor([-9, 20, 1000], dtype=torch.int32, device=device())
    near = torch.tensor([0, 20, 50], dtype=torch.int32, device=device())
    got = binding.attention(c.q, c.k, c.v, cu_seqlens=far)
    want = binding.attention(c.q, c.k, c.v, cu_seqlens=near)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = binding.attention_backward(c.dout, c.q, c.k, c.v, *want, cu_seqlens=far)
    want = binding.attention_backward(c.dout, c.q, c.k, c.v, *want, cu_seqlens=near)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("heads", [2, 64])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nothing_passes_between_sequences(heads, bad):
    """A sequence's results do not depend on another's values, finite or not."""
    import torch
    c = Case(6, [90, 70, 101], hq=heads, hk=heads, d=64, layout="dense")
    out, lse = call(c)
    grads = call_backward(c, out, lse)
    for t in (c.q, c.k, c.v, c.dout):
        t[90:160] = bad
    out2, lse2 = call(c)
    grads2 = call_backward(c, out2, lse2)
    for a, b in zip((out, *grads), (out2, *grads2)):
        assert torch.equal(a[:90], b[:90]) and torch.equal(a[160:], b[160:])
    assert torch.equal(lse[:, :90], lse2[:, :90]) and torch.equal(lse[:, 160:], lse2[:, 160:])


@pytest.mark.parametrize("heads", [2, 64])
def test_writes_stay_inside(heads):
    """Outputs in the layout of the inputs, with everything around them kept."""
    import torch
    c = Case(7, [77, 100], first=2, tail=3, hq=heads, hk=heads // 2, d=48)
    plain = call(c)
    grads = call_backward(c, *plain)
    dq, dk, dv = c.views(SENTINEL)
    buf = c.buffer
    call_backward(c, *plain, dq=dq, dk=dk, dv=dv)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, (dq, dk, dv)))
    assert bool((buf[:, -4:] == SENTINEL).all())
    wide = torch.full((c.T + 2, heads + 1, 52), SENTINEL, device=device())
    out = wide[1:-1, :heads, :48]
    call(c, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, plain[0])
    wide[1:-1, :heads, :48] = SENTINEL
    assert bool((wide == SENTINEL).all())
    # out over q
    q = c.q.clone()
    c.q = q
    got, _ = call(c, out=q)
    assert got is q and torch.equal(q, plain[0])


@pytest.mark.parametrize("hq,hk,tokens", [(4, 2, 300), (64, 16, 700), (128, 128, 600)])
def test_out_over_q_inside_the_projection(hq, hk, tokens):
    """out over the query columns of the buffer that holds the keys and values too."""
    import torch
    lengths = [tokens] if hq < 100 else [tokens // 6] * 6
    c = Case(hq, lengths, tail=5, hq=hq, hk=hk, d=64)
    want = call(c)
    keys, values = c.k.clone(), c.v.clone()
    got = call(c, out=c.q)
    assert got[0] is c.q and torch.equal(c.q, want[0]) and torch.equal(got[1], want[1])
    for kept, now in ((keys, c.k), (values, c.v)):
        assert torch.equal(kept[:tokens], now[:tokens]) and bool(now[tokens:].isnan().all())


def test_heads_of_three_tensors_in_turn():
    """Queries, keys and values of each head side by side, as some projections
    lay them out: inputs and gradients as views of such buffers, and a layout
    whose views do share elements refused."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    T, H, d = 90, 5, 32
    buf = torch.randn((T, H, 3, d), device=device())
    q, k, v = buf.unbind(2)
    out, lse = binding.attention(q, k, v)
    do = torch.randn_like(out)
    want = binding.attention_backward(do, *(x.contiguous() for x in (q, k, v)), out, lse)
    grad = torch.full((T, H, 3, d), SENTINEL, device=device())
    dq, dk, dv = grad.unbind(2)
    binding.attention_backward(do, q, k, v, out, lse, dq=dq, dk=dk, dv=dv)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), want))
    near = grad.view(T, -1)[:, 16:16 + (H - 1) * 3 * d + d].as_strided((T, H, d), (H * 3 * d, 3 * d, 1))
    with pytest.raises(binding.GemmError) as e:
        binding.attention_backward(do, q, k, v, out, lse, dq=near, dk=dk, dv=dv)
    assert e.value.status == -5


def test_offsets_past_32_bits():
    """Rows 16 K values apart, past 8 GiB into the buffer: sampled tiles of a windowed sequence."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    T, st, d, w = 140000, 16384, 32, 8
    buf = torch.empty((T, st), device=device())
    g = torch.Generator(device=device())
    g.manual_seed(1)
    small = torch.randn((T, 4 * d), generator=g, device=device())
    buf[:, 64:64 + 4 * d] = small
    q, k, v, do = (buf[:, 64 + i * d:64 + (i + 1) * d].unflatten(1, (1, d)) for i in range(4))
    out, lse = binding.attention(q, k, v, window=w)
    dense = [x.contiguous() for x in (q, k, v, do)]
    out2, lse2 = binding.attention(*dense[:3], window=w)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    a = binding.attention_backward(do, q, k, v, out, lse, window=w)
    b = binding.attention_backward(dense[3], *dense[:3], out, lse, window=w)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    rows = slice(T - 200, T)
    ro, _, eo, _ = OA.attention(*[x[rows].cpu().numpy() for x in dense[:3]], window=w)
    res = OA.compare(out[rows][w:].cpu().numpy(), ro[w:], eo[w:])
    assert res["fails"] == 0, res
    del buf, a, b, q, k, v, do
    torch.cuda.empty_cache()


def test_many_rows():
    """Three million rows: row numbers, tile numbers and offsets far past any
    other test's, sampled against the oracle at both ends."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    T, d, w = 3000000, 32, 8
    g = torch.Generator(device=device())
    g.manual_seed(2)
    q, k, v, do = (torch.randn((T, 1, d), generator=g, device=device()) for _ in range(4))
    out, lse = binding.attention(q, k, v, window=w)
    grads = binding.attention_backward(do, q, k, v, out, lse, window=w)
    for rows in (slice(0, 120), slice(T - 120, T)):
        host = [x[rows].cpu().numpy() for x in (do, q, k, v, out)]
        keep = slice(0, 120 - w) if rows.start == 0 else slice(w, 120)   # rows whose neighbours are all here
        ro, _, eo, _ = OA.attention(*host[1:4], window=w)
        res = OA.compare(host[4][keep], ro[keep], eo[keep])
        assert res["fails"] == 0, res
        want = OA.attention_backward(*host, lse[:, rows].cpu().numpy(), window=w)
        for y, ref, err in zip(grads, want[:3], want[3:]):
            res = OA.compare(y[rows][keep].cpu().numpy(), ref[keep], err[keep])
            assert res["fails"] == 0, res


def wide_case(seed):
    """More workgroups than one launch takes, nearly all with rows of their
    own: 65535 heads by 300 sequences of one or two rows."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    g = torch.Generator(device=device())
    g.manual_seed(seed)
    cu = cu_of([1, 2] * 150, first=1)
    T, H, d = int(cu[-1]) + 2, 65535, 4
    q, k, v, do = (torch.randn((T, H, d), generator=g, device=device()) for _ in range(4))
    return binding, cu, to_dev(cu), q, k, v, do


def test_more_workgroups_than_one_launch_takes():
    """Every part of the grid is done: the same bits as calls over fewer heads."""
    import torch
    binding, cu, dcu, q, k, v, _ = wide_case(1)
    out, lse = binding.attention(q, k, v, cu_seqlens=dcu)
    for at in range(0, q.shape[1], 8000):
        some = slice(at, min(at + 8000, q.shape[1]))
        o2, l2 = binding.attention(*(x[:, some].contiguous() for x in (q, k, v)), cu_seqlens=dcu)
        assert torch.equal(out[:, some], o2) and torch.equal(lse[some], l2)
    some = slice(65532, 65535)
    ro, rl, eo, el = OA.attention(*(x[:, some].cpu().numpy() for x in (q, k, v)), cu=cu)
    for y, ref, err in ((out[:, some], ro, eo), (lse[some], rl, el)):
        res = OA.compare(y.cpu().numpy(), ref, err)
        assert res["fails"] == 0, res


def test_gradients_of_more_workgroups_than_one_launch_takes():
    import torch
    binding, cu, dcu, q, k, v, do = wide_case(2)
    out, lse = binding.attention(q, k, v, cu_seqlens=dcu)
    grads = binding.attention_backward(do, q, k, v, out, lse, cu_seqlens=dcu)
    for at in range(0, q.shape[1], 8000):
        some = slice(at, min(at + 8000, q.shape[1]))
        part = [x[:, some].contiguous() for x in (do, q, k, v, out)]
        got = binding.attention_backward(*part, lse[some].contiguous(), cu_seqlens=dcu)
        assert all(torch.equal(a[:, some], b) for a, b in zip(grads, got))
    some = slice(65532, 65535)
    want = OA.attention_backward(*(x[:, some].cpu().numpy() for x in (do, q, k, v, out)), lse[some].cpu().numpy(), cu=cu)
    for y, ref, err in zip(grads, want[:3], want[3:]):
        res = OA.compare(y[:, some].cpu().numpy(), ref, err)
        assert res["fails"] == 0, res


def test_more_rows_than_one_launch_takes():
    """2^28 and more rows over all heads, so that the kernel in front of the
    backward pass needs slices too: sampled heads at both ends of the rows."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    T, H, d, w = 4100, 65535, 4, 2
    g = torch.Generator(device=device())
    g.manual_seed(3)
    q, k, v, do = (torch.randn((T, H, d), generator=g, device=device()) for _ in range(4))
    out, lse = binding.attention(q, k, v, window=w)
    assert binding.load_library().attn_backward_workspace_bytes(
        binding._PROBLEM.pack(0, 0, T, H, H, d, 1, w, 0.5)) == 4 * T * H
    grads = binding.attention_backward(do, q, k, v, out, lse, window=w)
    for heads in (slice(0, 2), slice(32767, 32769), slice(65533, 65535)):
        for rows in (slice(0, 100), slice(T // 2 - 50, T // 2 + 50), slice(T - 100, T)):
            host = [x[rows, heads].cpu().numpy() for x in (do, q, k, v, out)]
            # rows whose neighbours are all here
            keep = slice(0 if rows.start == 0 else w, 100 if rows.stop == T else 100 - w)
            ro, _, eo, _ = OA.attention(*host[1:4], window=w)
            res = OA.compare(host[4][keep], ro[keep], eo[keep])
            assert res["fails"] == 0, res
            want = OA.attention_backward(*host, lse[heads, rows].cpu().numpy(), window=w)
            for y, ref, err in zip(grads, want[:3], want[3:]):
                res = OA.compare(y[rows, heads].cpu().numpy()[keep], ref[keep], err[keep])
                assert res["fails"] == 0, res
    del q, k, v, do, out, grads
    torch.cuda.empty_cache()


def test_broadcast_views():
    """Key/value heads that are one tensor seen several times are read like
    any others; rows that are one row seen several times are refused, and so
    are outputs of either kind."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    r = torch.randn((50, 1, 64), device=device())
    q = torch.randn((50, 4, 64), device=device())
    k = r.expand(50, 4, 64)
    out, lse = binding.attention(q, k, k)
    want = binding.attention(q, k.contiguous(), k.contiguous())
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    got = binding.attention_backward(q, q, k, k, out, lse)
    want = binding.attention_backward(q, q, k.contiguous(), k.contiguous(), out, lse)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    rows = torch.randn((1, 4, 64), device=device()).expand(50, 4, 64)
    for call_it in (lambda: binding.attention(rows, k, k), lambda: binding.attention(q, k, k, out=rows),
                    lambda: binding.attention_backward(rows, q, k, k, out, lse),
                    lambda: binding.attention_backward(q, q, k, k, out, lse, dk=torch.empty_like(r).expand(50, 4, 64))):
        with pytest.raises(binding.GemmError) as e:
            call_it()
        assert e.value.status == -2
    # one token has no stride between tokens
    one = torch.randn((4, 64), device=device()).as_strided((1, 4, 64), (0, 64, 1))
    out, lse = binding.attention(one, one, one)
    assert torch.allclose(out, one) and bool(torch.isfinite(lse).all())
    grads = binding.attention_backward(one, one, one, one, out, lse)
    # a single key: the probability is 1 whatever the scores
    assert torch.allclose(grads[2], one) and float(grads[0].abs().max()) < 1e-5


def test_refusals_on_the_device():
    """Views that cannot be taken in 16-byte pieces, and results over inputs."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    buf = torch.randn((20, 4 * 64 + 2), device=device())
    odd = buf[:, 1:257].unflatten(1, (4, 64))              # base and token stride off
    q = odd.contiguous()
    for bad, status in ((lambda: binding.attention(odd, q, q), -3), (lambda: binding.attention(q, q, q, out=q), -5),
                        (lambda: binding.attention(q, q.clone(), q.clone(), scale=0.0), -4),
                        (lambda: binding.attention(q[..., :62], q[..., :62], q[..., :62]), -2)):
        with pytest.raises(binding.GemmError) as e:
            bad()
        assert e.value.status == status
    with pytest.raises(ValueError):
        binding.attention(q, q.cpu(), q)
    with pytest.raises(TypeError):
        binding.attention(q.double(), q, q)
    with pytest.raises(ValueError):
        binding.attention(q.transpose(1, 2), q.transpose(1, 2), q.transpose(1, 2))


def test_both_passes_refuse_a_problem_alike():
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    q = torch.randn((20, 2, 64), device=device())
    k, v, out, lse = q.clone(), q.clone(), q.clone(), torch.zeros((2, 20), device=device())
    for kw, width, status in (({"scale": 0.0}, 64, -4), ({"scale": float("inf")}, 64, -4), ({}, 62, -2)):
        for run in (lambda x: binding.attention(*(t[..., :x] for t in (q, k, v)), **kw),
                    lambda x: binding.attention_backward(*(t[..., :x] for t in (out, q, k, v, out)), lse, **kw)):
            with pytest.raises(binding.GemmError) as e:
                run(width)
            assert e.value.status == status


@pytest.mark.parametrize("heads", [2, 64])
def test_repeated_calls_give_the_same_bits(heads):
    import torch
    c = Case(8, [211, 90], hq=heads, hk=heads // 2, d=64)
    out, lse = call(c)
    grads = call_backward(c, out, lse)
    for _ in range(3):
        o2, l2 = call(c)
        g2 = call_backward(c, out, lse)
        assert torch.equal(out, o2) and torch.equal(lse, l2) and all(torch.equal(a, b) for a, b in zip(grads, g2))


def test_streams_and_graphs():
    """Calls queued on two streams at once, and two captured graphs replayed
    in turn with eager calls between, give the eager bits."""
    import torch
    cases = [Case(10 + i, [200, 50 + i], hq=4, hk=2, d=64) for i in range(2)]

    def step(c):
        out, lse = call(c)
        return (out, lse, *call_backward(c, out, lse))

    want = [step(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(4):
        got = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(step(c))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    graphs, held = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(step(c))
        graphs.append(g)
    for turn in range(3):
        for c in cases:
            c.q.mul_(1.25)
        fresh = [step(c) for c in cases]
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip(fresh, held):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), turn


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("plan", PLANS)
def test_verification_build(plan, d, monkeypatch):
    """The shipping library against the build with fences and full waits
    around the rows staged in LDS (heads of up to 64): the same bits."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    c = Case(d, d=d, **PLANS[plan])
    out, lse = call(c)
    got = (out, lse, *call_backward(c, out, lse))
    monkeypatch.setattr(binding, "_lib", binding.load_sync_check_library())
    want = (*call(c), *call_backward(c, out, lse))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
