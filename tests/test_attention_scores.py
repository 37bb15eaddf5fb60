"""Attention with capped, biased and prefix-masked scores on the GPU, forward
and backward, against the oracle (oracle/attention.py): every head width and
way of dealing out rows, each form by itself and together, with windows and
shared heads, prefixes that end anywhere or past their sequence, caps from
ones that nothing reaches to ones that all scores pass, many sequences,
strided views, poisoned neighbours, other streams and graph replays.  The
bounds are the oracle's, counted per element."""
import numpy as np
import pytest

from oracle import attention as OA

from _gpu import device, say, to_dev

pytestmark = pytest.mark.gpu

SENTINEL = -777.0
# the forms, as functions of the number of heads and the sequences' lengths
SLOPES = lambda h: (2.0 ** (-8.0 * (1 + np.arange(h)) / h)).astype(np.float32)  # noqa: E731


def forms(name, hq, lengths, r):
    form = {}
    if name in ("cap", "all", "cap+prefix"):
        form["softcap"] = 2.5
    if name in ("slopes", "all"):
        form["slopes"] = SLOPES(hq) * np.where(np.arange(hq) % 3 == 2, -0.1, 1.0).astype(np.float32)
    if name in ("prefix", "all", "cap+prefix"):
        form["prefix"] = np.array([r.integers(0, n + 1) if n else 3 for n in lengths], dtype=np.int32)
    return form


class Case:
    """Device tensors of a call: q, k, v as views of one projection's output,
    everything around them and in the rows of no sequence NaN."""

    def __init__(self, seed, lengths, form, first=0, tail=0, hq=2, hk=1, d=64, window=0, causal=True, scale=None,
                 gain=2.0):
        import torch
        r = np.random.default_rng(seed)
        if isinstance(form, str):
            form = forms(form, hq, lengths, r)
        self.form = form
        self.T = T = first + sum(lengths) + tail
        self.kw = {"window": window, "causal": causal, "scale": scale}
        self.cu = None if list(lengths) == [T] else np.cumsum([first, *lengths]).astype(np.int32)
        self.shapes = ((T, hq, d), (T, hk, d), (T, hk, d))
        self.host = [(r.standard_normal(s) * g).astype(np.float32) for s, g in zip(self.shapes, (gain, 1.0, 1.0))]
        self.g = r.standard_normal(self.shapes[0]).astype(np.float32)
        self.used = np.zeros(T, bool)
        for a, b in OA.sequences(self.cu, T):
            self.used[a:b] = True
        w = [s[1] * d for s in self.shapes]
        buf = torch.full((T, sum(w) + 4), float("nan"), device=device())
        rows = to_dev(np.flatnonzero(self.used))
        buf[rows, :-4] = torch.cat([to_dev(x[self.used].reshape(-1, n)) for x, n in zip(self.host, w)], 1)
        self.q, self.k, self.v = (x.unflatten(1, s[1:]) for x, s in zip(buf[:, :-4].split(w, 1), self.shapes))
        self.dout = torch.full(self.shapes[0], float("nan"), device=device())
        self.dout[rows] = to_dev(self.g[self.used])
        self.dev = {"cu_seqlens": None if self.cu is None else to_dev(self.cu), "softcap": form.get("softcap", 0.0),
                    "slopes": to_dev(form["slopes"]) if "slopes" in form else None,
                    "prefix_lens": to_dev(form["prefix"]) if "prefix" in form else None}

    def clean(self, a):
        return np.where(self.used[:, None, None], a, 0.0)

    def oracle_args(self):
        return [self.clean(x) for x in self.host], {"cu": self.cu, **self.kw, **self.form}


def call(c, **kw):
    from tiled_dense_gemm_matmul_amd import binding
    return binding.attention(c.q, c.k, c.v, **c.kw, **c.dev, **kw)


def call_backward(c, out, lse, **kw):
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    if "slopes" in c.form and "dslopes" not in kw:
        kw["dslopes"] = torch.empty_like(c.dev["slopes"])
    return binding.attention_backward(c.dout, c.q, c.k, c.v, out, lse, **c.kw, **c.dev, **kw)


def close(label, name, y, ref, err):
    res = OA.compare(y.cpu().numpy(), ref, err)
    say(f"  {label} {name}: max err/bound {res['max_ratio']:.3g}, fails {res['fails']} of {res['n']}")
    assert res["fails"] == 0, (label, name, res)


def check(c, label):
    say(label)
    out, lse = call(c)
    args, kw = c.oracle_args()
    ro, rl, eo, el = OA.scored_attention(*args, **kw)
    close(label, "out", out, ro, eo)
    close(label, "lse", lse, rl, el)
    got = call_backward(c, out, lse)
    assert len(got) == (4 if "slopes" in c.form else 3)
    want = OA.scored_attention_backward(c.clean(c.g), *args, out.cpu().numpy(), lse.cpu().numpy(), **kw)
    for i, y in enumerate(got):
        close(label, ("dq", "dk", "dv", "dslopes")[i], y, want[i], want[4 + i])


FORMS = ["cap", "slopes", "prefix", "all"]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("d", [4, 20, 32, 48, 64, 80, 96, 100, 128])
def test_head_widths(d, form):
    check(Case(d, [70, 33], form, hq=2, hk=1, d=d), f"scores D={d} {form}")


# one problem for each way the kernels deal out rows and keys: few rows, many
# rows, shared heads, and many short sequences
PLANS = {"few": dict(lengths=[900], hq=8, hk=8), "many": dict(lengths=[520], tail=3, hq=64, hk=64),
         "shared": dict(lengths=[300, 33], hq=32, hk=2),
         "short": dict(lengths=[200, 1, 0, 130, 120, 77], first=2, tail=9, hq=128, hk=128)}


@pytest.mark.parametrize("d", [20, 32, 64, 96, 128])
@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("form,window", [("all", 0), ("all", 70), ("cap+prefix", 0)])
def test_plans(plan, d, form, window):
    check(Case(d, form=form, d=d, window=window, **PLANS[plan]), f"scores {plan} D={d} {form} window {window}")


@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("form", FORMS)
def test_results_inside_one_buffer(plan, form):
    """out over q inside the projection's output, and the gradients as columns
    of one buffer, have the bits of results of their own; what lies beside
    them stays."""
    import torch
    c = Case(6, form=form, d=64, **PLANS[plan])
    out, lse = call(c)
    want = call_backward(c, out, lse)
    w = [s[1] * s[2] for s in c.shapes]
    buf = torch.full((c.T, sum(w) + 4), SENTINEL, device=device())
    views = [x.unflatten(1, s[1:]) for x, s in zip(buf[:, :-4].split(w, 1), c.shapes)]
    got = call_backward(c, out, lse, dq=views[0], dk=views[1], dv=views[2])
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert bool((buf[:, -4:] == SENTINEL).all())
    k, v = c.k.clone(), c.v.clone()
    over, lse2 = call(c, out=c.q)
    assert over.data_ptr() == c.q.data_ptr() and torch.equal(over, out) and torch.equal(lse2, lse)
    assert torch.equal(c.k.view(torch.int32), k.view(torch.int32))
    assert torch.equal(c.v.view(torch.int32), v.view(torch.int32))


@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("form", ["cap", "slopes"])
def test_both_ways(plan, form):
    """Without a causal mask: distances ahead count as those behind."""
    check(Case(5, form=form, d=64, causal=False, **PLANS[plan]), f"scores both ways {plan} {form}")


@pytest.mark.parametrize("lengths", [[1], [2], [15], [16], [17], [64], [65], [1] * 40, [0, 5, 0, 0, 3, 0], [127, 129],
                                     [513], list(range(1, 24))])
@pytest.mark.parametrize("window", [0, 5])
def test_lengths(lengths, window):
    check(Case(len(lengths), lengths, "all", hq=3, hk=3, d=32, window=window), f"scores {str(lengths)[:30]}")


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 31, 32, 33, 100, 199, 200, 201, 1 << 30, -1, -(1 << 31)])
@pytest.mark.parametrize("hq", [2, 128])
def test_prefixes(prefix, hq):
    """Prefixes that end anywhere in a tile, past the sequence and before it."""
    form = {"prefix": np.array([prefix, 7, prefix], dtype=np.int32)}
    check(Case(3, [200, 50, 130], form, hq=hq, hk=hq, d=32, first=1, tail=2), f"scores prefix {prefix} heads {hq}")


def test_prefix_of_one_sequence_without_bounds():
    check(Case(3, [150], {"prefix": np.array([60], dtype=np.int32)}, hq=4, hk=2, d=64), "scores one prefix")


@pytest.mark.parametrize("heads", [2, 64])
def test_whole_prefixes_and_none_give_the_masks_they_are(heads):
    """A prefix as long as its sequence is no causal mask, one of none is the causal mask."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    c = Case(4, [90, 70], {"prefix": np.array([90, 70], dtype=np.int32)}, hq=heads, hk=heads, d=64)
    dcu = c.dev["cu_seqlens"]
    for lens, causal in (([90, 70], False), ([0, 0], True)):
        c.dev["prefix_lens"] = torch.tensor(lens, dtype=torch.int32, device=device())
        out, lse = call(c)
        ro, rl = binding.attention(c.q, c.k, c.v, cu_seqlens=dcu, causal=causal)
        # scores through one product more, of the same order of roundings
        assert torch.allclose(out, ro, rtol=1e-4, atol=1e-5) and torch.allclose(lse, rl, rtol=1e-5, atol=1e-5)
        got = call_backward(c, ro, rl)
        want = binding.attention_backward(c.dout, c.q, c.k, c.v, ro, rl, cu_seqlens=dcu, causal=causal)
        assert all(torch.allclose(a, b, rtol=1e-3, atol=1e-4) for a, b in zip(got, want))


@pytest.mark.parametrize("softcap,gain", [(1e-6, 1.0), (1e-3, 1.0), (0.7, 2.0), (2.0, 2.0), (8.0, 4.0), (30.0, 1.0),
                                          (30.0, 60.0), (1e6, 1.0), (1e6, 1e4), (50.0, 1e10), (50.0, 1e-10)])
@pytest.mark.parametrize("d", [32, 64])
def test_caps(softcap, gain, d):
    """Scores far below the cap, about it, and all past it."""
    check(Case(9, [150, 40], {"softcap": softcap}, hq=2, hk=2, d=d, gain=gain), f"scores cap {softcap} gain {gain}")


def test_infinite_products_are_capped():
    """A product past fp32's range is the cap, of either sign, and its gradient is zero."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    q = torch.full((3, 1, 32), 1e30, device=device())
    k = torch.full((3, 1, 32), 1e30, device=device())
    k[1] = -1e30
    v = torch.randn((3, 1, 32), device=device())
    out, lse = binding.attention(q, k, v, softcap=2.0, causal=False)
    w = torch.softmax(torch.tensor([2.0, -2.0, 2.0], dtype=torch.float64, device=device()), 0)
    want = (w[:, None] * v[:, 0].double()).sum(0)
    assert torch.allclose(out[:, 0].double(), want.expand(3, 32), rtol=1e-5, atol=1e-6)
    dq, dk, dv = binding.attention_backward(v, q, k, v, out, lse, softcap=2.0, causal=False)
    assert not dq.any() and not dk.any() and bool(torch.isfinite(dv).all())


@pytest.mark.parametrize("slope", [0.0, 1e-8, 0.5, 100.0, -0.01, 1e5])
@pytest.mark.parametrize("hq", [2, 128])
def test_slopes(slope, hq):
    """Slopes from none to ones that leave a row its own key, and growing ones."""
    check(Case(8, [200, 77], {"slopes": np.full(hq, slope, np.float32)}, hq=hq, hk=hq // 2, d=32),
          f"scores slope {slope} heads {hq}")


def test_a_single_key_has_probability_one():
    """Rows that see themselves alone.  The sum of exponentials is exp2 of what
    the score's product with log2(e) was rounded by, a number next to 1 that is
    rounded by 2^-24, and its logarithm less that difference, times ln 2, is
    off by less than 2^-23: so is lse, and dv is off by less than 2^-22 of
    dout.  From scores of 8 on, whose half a step is 2^-21, lse is the final
    score itself and dv is dout to the bit."""
    import torch
    seen = 0
    for T, heads in ((40, 1), (1024, 32), (128, 512)):
        for form in ({"softcap": 3.0}, {"slopes": np.ones(heads, np.float32)}, {"softcap": 300.0}):
            c = Case(2, [T], form, hq=heads, hk=heads, d=32, window=1, gain=20.0)
            out, lse = call(c)
            assert torch.allclose(out, c.v, rtol=1e-6, atol=0)
            dv = call_backward(c, out, lse)[2]
            assert bool(((dv - c.dout).abs() <= 2.0 ** -22 * c.dout.abs()).all())
            large = lse.t().abs() >= 8
            assert torch.equal(dv[large], c.dout[large])
            seen += int(large.sum())
    assert seen > 1000


@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 1), (6, 2), (16, 2), (200, 50)])
def test_shared_heads(hq, hk):
    check(Case(hq, [200, 57], "all", first=1, tail=5, hq=hq, hk=hk, d=64, window=90), f"scores heads {hq}/{hk}")


@pytest.mark.parametrize("number,heads", [(300, 2), (300, 64), (512, 2), (513, 2), (4097, 2)])
def test_many_sequences(number, heads):
    """On both sides of the number from which a tile's sequence is searched for: each has its own prefix."""
    r = np.random.default_rng(number)
    lengths = [int(n) for n in r.choice(6, number)]
    lengths[7], lengths[number // 2], lengths[number - 2] = 90, 150, 40
    check(Case(number, lengths, "all", first=5, tail=3, hq=heads, hk=heads, d=32), f"scores {number} sequences")


def test_nothing_passes_between_sequences():
    import torch
    for heads in (2, 64):
        c = Case(6, [90, 70, 101], "all", hq=heads, hk=heads, d=64)
        out, lse = call(c)
        grads = call_backward(c, out, lse)
        for bad in (float("nan"), float("inf")):
            for t in (c.q, c.k, c.v, c.dout):
                t[90:160] = bad
            out2, lse2 = call(c)
            grads2 = call_backward(c, out2, lse2)
            for a, b in zip((out, *grads[:3]), (out2, *grads2[:3])):
                assert torch.equal(a[:90], b[:90]) and torch.equal(a[160:], b[160:])
            assert torch.equal(lse[:, :90], lse2[:, :90]) and torch.equal(lse[:, 160:], lse2[:, 160:])


def test_empty():
    """No tokens, and no sequence: zero gradients of the slopes."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    dev = device()
    sl, ds = torch.ones(2, device=dev), torch.full((2,), 9.0, device=dev)
    q = torch.empty((0, 2, 32), device=dev)
    out, lse = binding.attention(q, q, q, slopes=sl, softcap=3.0)
    got = binding.attention_backward(q, q, q, q, out, lse, slopes=sl, dslopes=ds)
    assert out.shape == (0, 2, 32) and got[3] is ds and not ds.any()
    for n in (0, 5):
        q = torch.full((37, 2, 32), float("nan"), device=dev)
        cu = torch.zeros(n + 1, dtype=torch.int32, device=dev)
        pre = torch.ones(n, dtype=torch.int32, device=dev)
        ds.fill_(9.0)
        out, lse = binding.attention(q, q, q, cu_seqlens=cu, slopes=sl, prefix_lens=pre)
        grads = binding.attention_backward(q, q, q, q, q, lse, cu_seqlens=cu, slopes=sl, prefix_lens=pre, dslopes=ds)
        assert not out.any() and bool((lse == -float("inf")).all()) and not any(bool(x.any()) for x in grads)


def test_writes_stay_inside():
    import torch
    for heads in (2, 64):
        c = Case(7, [77, 100], "all", first=2, tail=3, hq=heads, hk=heads // 2, d=48)
        plain = call(c)
        grads = call_backward(c, *plain)
        w = [s[1] * s[2] for s in c.shapes]
        buf = torch.full((c.T, sum(w) + 8), SENTINEL, device=device())
        dq, dk, dv = (x.unflatten(1, s[1:]) for x, s in zip(buf[:, 4:-4].split(w, 1), c.shapes))
        ds = torch.full((heads + 8,), SENTINEL, device=device())
        got = call_backward(c, *plain, dq=dq, dk=dk, dv=dv, dslopes=ds[4:-4])
        assert all(torch.equal(a, b) for a, b in zip(grads, got))
        assert bool((buf[:, :4] == SENTINEL).all()) and bool((buf[:, -4:] == SENTINEL).all())
        assert bool((ds[:4] == SENTINEL).all()) and bool((ds[-4:] == SENTINEL).all())
        wide = torch.full((c.T + 2, heads + 1, 52), SENTINEL, device=device())
        call(c, out=wide[1:-1, :heads, :48])
        assert torch.equal(wide[1:-1, :heads, :48], plain[0])
        wide[1:-1, :heads, :48] = SENTINEL
        assert bool((wide == SENTINEL).all())
        got, _ = call(c, out=c.q)                      # out over q, inside the projection
        assert got is c.q and torch.equal(c.q, plain[0])


def test_without_the_slopes_gradient():
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    c = Case(3, [600], "all", hq=8, hk=4, d=64)
    out, lse = call(c)
    want = call_backward(c, out, lse)
    got = binding.attention_backward(c.dout, c.q, c.k, c.v, out, lse, **c.kw, **c.dev)
    assert len(got) == 3 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_slopes_by_differences():
    """The slopes' gradient against central differences of the forward pass in 64 bits."""
    c = Case(11, [60, 33], "all", hq=4, hk=2, d=32)
    out, lse = call(c)
    got = call_backward(c, out, lse)[3].cpu().numpy()
    args, kw = c.oracle_args()
    for h in range(4):
        def at(e):
            moved = kw["slopes"].astype(np.float64)
            moved[h] += e
            return (OA.scored_attention(*args, **{**kw, "slopes": moved})[0] * c.clean(c.g)).sum()
        slope = (at(1e-5) - at(-1e-5)) / 2e-5
        assert abs(slope - got[h]) < 1e-4 * max(1.0, abs(slope))


def test_long_sequence():
    """Rows past 2^14, where a window leaves the bias its far distances out of sight: sampled rows at both ends."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    T, d, w = 300000, 32, 40
    g = torch.Generator(device=device())
    g.manual_seed(2)
    q, k, v, do = (torch.randn((T, 1, d), generator=g, device=device()) for _ in range(4))
    sl = torch.full((1,), 0.03, device=device())
    kw = {"window": w, "softcap": 2.0, "slopes": sl}
    out, lse = binding.attention(q, k, v, **kw)
    grads = binding.attention_backward(do, q, k, v, out, lse, **kw, dslopes=torch.empty_like(sl))
    host_kw = {"window": w, "softcap": 2.0, "slopes": [float(sl[0])]}
    total = 0.0
    for rows in (slice(0, 300), slice(T - 300, T)):
        host = [x[rows].cpu().numpy() for x in (do, q, k, v, out)]
        keep = slice(0, 300 - w) if rows.start == 0 else slice(w, 300)
        ro, _, eo, _ = OA.scored_attention(*host[1:4], **host_kw)
        close("long", "out", out[rows][keep], ro[keep], eo[keep])
        want = OA.scored_attention_backward(*host, lse[:, rows].cpu().numpy(), **host_kw)
        for i in range(3):
            close("long", "dqdkdv", grads[i][rows][keep], want[i][keep], want[4 + i][keep])
    # the slope's gradient over all rows, in 64 bits over diagonals
    q, k, v, do, out = (x[:, 0].double() for x in (q, k, v, do, out))
    delta, l, size = (do * out).sum(1), lse[0].double(), 0.0
    for m in range(1, w):
        s = 2.0 * torch.tanh((q[m:] * k[:-m]).sum(1) / d ** 0.5 / 2.0) - float(sl[0]) * m
        part = m * torch.exp(s - l[m:]) * ((do[m:] * v[:-m]).sum(1) - delta[m:])
        total, size = total - part.sum(), size + part.abs().sum()
    # each term is off by some 200 u (its score, lse, two sums of 32 products), the sum far less
    assert abs(float(total) - float(grads[3])) < 200 * 2.0 ** -24 * float(size)


def test_more_workgroups_than_one_launch_takes():
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    g = torch.Generator(device=device())
    g.manual_seed(1)
    lengths = [1, 2] * 150
    cu = to_dev(np.cumsum([1, *lengths]).astype(np.int32))
    T, H, d = int(cu[-1]) + 2, 65535, 4
    q, k, v = (torch.randn((T, H, d), generator=g, device=device()) for _ in range(3))
    sl = torch.rand((H,), generator=g, device=device())
    pre = to_dev(np.arange(300, dtype=np.int32) % 3)
    kw = {"cu_seqlens": cu, "softcap": 1.5, "prefix_lens": pre}
    out, lse = binding.attention(q, k, v, slopes=sl, **kw)
    grads = binding.attention_backward(v, q, k, v, out, lse, slopes=sl, dslopes=torch.empty_like(sl), **kw)
    for at in range(0, H, 16000):
        some = slice(at, min(at + 16000, H))
        part = [x[:, some].contiguous() for x in (q, k, v)]
        o2, l2 = binding.attention(*part, slopes=sl[some].contiguous(), **kw)
        assert torch.equal(out[:, some], o2) and torch.equal(lse[some], l2)
        g2 = binding.attention_backward(part[2], *part, o2, l2, slopes=sl[some].contiguous(),
                                        dslopes=torch.empty_like(sl[some]), **kw)
        assert all(torch.equal(a[:, some], b) for a, b in zip(grads[:3], g2)) and torch.equal(grads[3][some], g2[3])
    del q, k, v, out, grads
    torch.cuda.empty_cache()


def test_refusals_on_the_device():
    import torch
    from tiled_dense_gemm_matmul_amd import binding as B
    dev = device()
    q = torch.randn((20, 4, 64), device=dev)
    k, v = q[:, :2].clone(), q[:, 2:].clone()
    out, lse = B.attention(q, k, v, softcap=5.0)
    sl, pre, cu = (torch.ones(4, device=dev), torch.ones(2, dtype=torch.int32, device=dev),
                   torch.tensor([0, 9, 20], dtype=torch.int32, device=dev))
    for bad in (lambda: B.attention(q, k, v, slopes=sl[:3]), lambda: B.attention(q, k, v, slopes=sl.cpu()),
                lambda: B.attention(q, k, v, slopes=sl.double()), lambda: B.attention(q, k, v, prefix_lens=pre),
                lambda: B.attention(q, k, v, cu_seqlens=cu, prefix_lens=pre[:1]),
                lambda: B.attention(q, k, v, cu_seqlens=cu, prefix_lens=pre, causal=False),
                lambda: B.attention_backward(out, q, k, v, out, lse, dslopes=sl),
                lambda: B.attention_backward(out, q, k, v, out, lse, slopes=sl, dslopes=sl[:2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        B.attention(q, k, v, cu_seqlens=cu, prefix_lens=pre.long())
    for cap in (-1.0, float("nan"), 1e7, 1e-9):
        for bad in (lambda: B.attention(q, k, v, softcap=cap),
                    lambda: B.attention_backward(out, q, k, v, out, lse, softcap=cap)):
            with pytest.raises(B.GemmError) as e:
                bad()
            assert e.value.status == -4
    with pytest.raises(B.GemmError) as e:
        B.attention_backward(out, q, k, v, out, lse, slopes=sl, dslopes=sl)
    assert e.value.status == -5


def test_repeated_calls_streams_and_graphs():
    """The same bits from repeated calls, from two streams at once, and from
    two captured graphs replayed in turn with eager calls between."""
    import torch
    cases = [Case(10 + i, [200, 50 + i], "all", hq=4, hk=2, d=64) for i in range(2)]
    cases.append(Case(20, [1500], "all", hq=8, hk=8, d=32))

    def step(c):
        out, lse = call(c)
        return (out, lse, *call_backward(c, out, lse))

    want = [step(c) for c in cases]
    for c, a in zip(cases, want):
        assert all(torch.equal(x, y) for x, y in zip(a, step(c)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
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
            c.dev["prefix_lens"].add_(1)
        fresh = [step(c) for c in cases]
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip(fresh, held):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), turn


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("plan", PLANS)
def test_verification_build(plan, d, monkeypatch):
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    c = Case(d, form="all", d=d, **PLANS[plan])
    out, lse = call(c)
    got = (out, lse, *call_backward(c, out, lse))
    monkeypatch.setattr(binding, "_lib", binding.load_sync_check_library())
    want = (*call(c), *call_backward(c, out, lse))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
