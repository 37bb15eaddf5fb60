"""qk_norm_rope and qk_norm_rope_backward on the GPU against the oracle
(oracle/attention.py): every lane layout of the kernels, 16-byte and 4-byte
accesses, both pairings, partly rotated heads, far positions, strided views
inside poisoned buffers, results over the inputs, and graph replays."""
import numpy as np
import pytest

from oracle import attention as OA

from _gpu import device, say, to_dev

pytestmark = pytest.mark.gpu

SENTINEL = -777.0


class Case:
    def __init__(self, seed, T, hq, hk, d, rotated, interleaved=False, first=0, wide=False, pad=0, gain=1.0):
        import torch
        r = np.random.default_rng(seed)
        self.shapes = ((T, hq, d), (T, hk, d))
        self.x = [(r.standard_normal(s) * gain).astype(np.float32) for s in self.shapes]
        self.g = [r.standard_normal(s).astype(np.float32) for s in self.shapes]
        self.w = [(1 + 0.1 * r.standard_normal(d)).astype(np.float32) for _ in range(2)]
        self.pos = (first + np.arange(T) * 3).astype(np.int64 if wide else np.int32)
        self.freq = (10000.0 ** (-np.arange(rotated // 2) / max(1, rotated // 2))).astype(np.float32)
        self.interleaved, self.pad = interleaved, pad
        self.q, self.k = self.views(self.x)
        self.gq, self.gk = self.views(self.g)
        self.common = tuple(to_dev(a) for a in (*self.w, self.pos, self.freq))
        torch.cuda.synchronize()

    def views(self, arrays, fill=float("nan")):
        """Both tensors as columns of one buffer, `pad` columns around each."""
        import torch
        T, d, p = self.shapes[0][0], self.shapes[0][2], self.pad
        w = [s[1] * d for s in self.shapes]
        self.buffer = buf = torch.full((T, sum(w) + 3 * p), fill, device=device())
        out = []
        at = p
        for n, s, a in zip(w, self.shapes, arrays or (None, None)):
            t = buf[:, at:at + n].unflatten(1, s[1:])
            if a is not None:
                t.copy_(to_dev(a))
            out.append(t)
            at += n + p
        return out

    def kept(self, fill):
        """Whether the columns around the last views() are untouched."""
        p, d = self.pad, self.shapes[0][2]
        a = p + self.shapes[0][1] * d
        cols = [self.buffer[:, :p], self.buffer[:, a:a + p], self.buffer[:, self.buffer.shape[1] - p:]]
        return all(bool((c == fill).all()) for c in cols)


def run(c, **kw):
    from tiled_dense_gemm_matmul_amd import binding
    return binding.qk_norm_rope(c.q, c.k, *c.common, interleaved=c.interleaved, **kw)


def run_backward(c, **kw):
    from tiled_dense_gemm_matmul_amd import binding
    return binding.qk_norm_rope_backward(c.gq, c.gk, c.q, c.k, *c.common, interleaved=c.interleaved, **kw)


def verify(c, got, grads, label):
    names, refs, errs, ys = [], [], [], []
    for i, n in enumerate("qk"):
        ref, err = OA.qk_norm_rope(c.x[i], c.w[i], c.pos, c.freq, 1e-6, c.interleaved)
        dx, dw, edx, edw = OA.qk_norm_rope_backward(c.g[i], c.x[i], c.w[i], c.pos, c.freq, 1e-6, c.interleaved)
        names += [n, "d" + n, f"d{n}_weight"]
        refs += [ref, dx, dw]
        errs += [err, edx, edw]
        ys += [got[i], grads[i], grads[2 + i]]
    for n, y, ref, err in zip(names, ys, refs, errs):
        res = OA.compare(y.cpu().numpy(), ref, err)
        say(f"  {label} {n}: max err/bound {res['max_ratio']:.3g}, fails {res['fails']} of {res['n']}")
        assert res["fails"] == 0, (label, n, res)


# head widths that fill each group of lanes, and ones that do not
@pytest.mark.parametrize("d,rotated", [(8, 8), (16, 16), (24, 8), (32, 32), (48, 16), (64, 64), (64, 32), (96, 96),
                                       (128, 128), (128, 16), (160, 64), (256, 256), (256, 0),
                                       # 4-byte accesses: pairs that four do not divide
                                       (2, 2), (6, 4), (12, 12), (20, 10), (64, 12), (100, 50), (130, 130), (254, 6)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_widths(d, rotated, interleaved):
    say(f"qk_norm_rope D={d} rotated={rotated} interleaved={interleaved}")
    c = Case(d + rotated, 19, 5, 2, d, rotated, interleaved, first=7, pad=4 if d % 4 == 0 else 1)
    verify(c, run(c), run_backward(c), f"D={d}/{rotated}")


@pytest.mark.parametrize("T,hq,hk", [(1, 1, 1), (1, 40, 8), (2, 3, 7), (513, 12, 12), (4100, 2, 1), (33, 130, 1)])
def test_sizes(T, hq, hk):
    say(f"qk_norm_rope T={T} heads {hq}+{hk}")
    c = Case(T, T, hq, hk, 64, 64, wide=True)
    verify(c, run(c), run_backward(c), f"T={T} {hq}+{hk}")


def test_long_weight_gradient():
    """Sums over 300 000 heads of each weight value stay as good as short ones."""
    c = Case(3, 20000, 12, 3, 32, 16)
    verify(c, run(c), run_backward(c), "long")


@pytest.mark.parametrize("first,wide", [(-5, False), (1 << 20, False), (2 ** 31 - 200, False), (1 << 33, True),
                                        (-(1 << 40), True)])
def test_far_positions(first, wide):
    c = Case(4, 40, 4, 1, 64, 64, first=first, wide=wide)
    verify(c, run(c), run_backward(c), f"from {first}")


def turned(pos, freq):
    """Cosine and sine of pos * freq in 64 bits, however near to their zeros:
    the angle's distance from the nearest quarter turn is formed in 60 digits."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    quarter = Decimal("3.14159265358979323846264338327950288419716939937510582097494459") / 2
    angle = Decimal(int(pos)) * Decimal(float(freq))
    n = int((angle / quarter).to_integral_value())
    rest = float(angle - n * quarter)
    c, s = np.cos(rest), np.sin(rest)
    return [(c, s), (-s, c), (-c, -s), (s, -c)][n % 4]


@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_near_quarter_turns(interleaved):
    """Sine and cosine are good to fp32 relative to themselves, next to their
    zeros too.  Heads hold (a, 0) in every pair, so a result is one product of
    the normed a, which position 0 gives as it is: u = 2^-24 for that product,
    4 u for sine and cosine, u each for the product and the sum that correct
    them by the angle's rest, and one to spare."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    r, d = np.random.default_rng(8), 256
    quarters = r.integers(1, 9, d // 2) * (np.pi / 2)
    freq = (quarters + r.choice([-1.0, 1.0], d // 2) * 2.0 ** -r.integers(1, 20, d // 2)).astype(np.float32)
    pos = np.array([0, 1, 3, -5, 1001, -123457, 2 ** 24 + 1, 10 ** 9 + 7, 2 ** 40 + 3], dtype=np.int64)
    first, second = OA._pairs(d, d, interleaved)
    x = np.zeros((len(pos), 1, d), np.float32)
    x[:, :, first] = 1.0 + r.random(d // 2).astype(np.float32)
    w = torch.ones(d, device=device())
    y, _ = binding.qk_norm_rope(to_dev(x), to_dev(x), w, w, to_dev(pos), to_dev(freq), interleaved=interleaved)
    y = y.cpu().numpy().astype(np.float64)[:, 0]
    n = y[0, first]
    assert not y[0, second].any()
    want = np.array([[turned(p, f) for f in freq] for p in pos])
    for name, got, ref in (("cosine", y[:, first] / n, want[..., 0]), ("sine", y[:, second] / n, want[..., 1])):
        far = np.abs(got - ref) / np.maximum(np.abs(ref), 1e-300)
        far[0] = 0.0 if name == "cosine" else np.where(got[0] == 0, 0.0, np.inf)
        say(f"  {name}: off by up to {far.max() * 2 ** 24:.3g} u")
        assert far.max() <= 8 * 2.0 ** -24, name


@pytest.mark.parametrize("pad", [1, 2, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_views_in_place_and_neighbours(pad, interleaved):
    """Strides and offsets of any alignment, results in views of one buffer
    and over the inputs, with everything around them kept."""
    import torch
    c = Case(5, 37, 6, 2, 64, 32, interleaved, pad=pad)
    got, grads = run(c), run_backward(c)
    verify(c, got, grads, f"pad {pad}")
    oq, ok = c.views(None, SENTINEL)
    run(c, q_out=oq, k_out=ok)
    assert torch.equal(oq, got[0]) and torch.equal(ok, got[1]) and c.kept(SENTINEL)
    oq, ok = c.views(None, SENTINEL)
    run_backward(c, dq=oq, dk=ok)
    assert torch.equal(oq, grads[0]) and torch.equal(ok, grads[1]) and c.kept(SENTINEL)
    # over the gradients, then over the inputs
    gq, gk = c.gq.clone(), c.gk.clone()
    c.gq, c.gk, keep = gq, gk, (c.gq, c.gk)
    again = run_backward(c, dq=gq, dk=gk)
    assert all(torch.equal(a, b) for a, b in zip(again, grads))
    c.gq, c.gk = keep
    q, k = c.q, c.k
    c.q, c.k = q.clone(), k.clone()
    again = run_backward(c, dq=c.q, dk=c.k)
    assert all(torch.equal(a, b) for a, b in zip(again, grads))
    c.q, c.k = q.clone(), k.clone()
    dense = run(c)             # the clones are dense: other accesses, another order of a row's sum
    again = run(c, q_out=c.q, k_out=c.k)
    assert torch.equal(c.q, dense[0]) and torch.equal(c.k, dense[1]) and again[0] is c.q
    verify(c, dense, grads, f"dense {pad}")


def test_small_values():
    """eps carries rows of zeros; a row of tiny values is normed with it."""
    import torch
    c = Case(6, 8, 2, 2, 64, 64, gain=1e-5)
    verify(c, run(c), run_backward(c), "tiny")
    c.q.zero_()
    got, grads = run(c), run_backward(c)
    assert not got[0].any() and bool(torch.isfinite(grads[0]).all()) and not grads[2].any()


def test_no_tokens():
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    dev = device()
    q, w = torch.empty((0, 2, 32), device=dev), torch.ones(32, device=dev)
    common = (w, w, torch.empty(0, dtype=torch.int32, device=dev), torch.ones(16, device=dev))
    assert binding.qk_norm_rope(q, q.clone(), *common)[0].shape == (0, 2, 32)
    grads = binding.qk_norm_rope_backward(q, q, q, q, *common, dq_weight=w.clone(), dk_weight=w.clone())
    assert not grads[2].any() and not grads[3].any()


def test_more_tokens_than_one_launch_takes():
    """A wave a token, past 2^26 tokens: the last ones get the bits of a call
    of their own."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    T, dev = (1 << 26) + 5, device()
    q, k = (torch.randn((T, 1, 2), device=dev) for _ in range(2))
    w, freq = torch.ones(2, device=dev), torch.full((1,), 0.25, device=dev)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    common = (w, w * 0.5)
    out = [torch.full_like(q, SENTINEL) for _ in range(2)]
    binding.qk_norm_rope(q, k, *common, pos, freq, q_out=out[0], k_out=out[1])
    grads = binding.qk_norm_rope_backward(q, k, q, k, *common, pos, freq)
    for a in (0, T // 2, T - 5000):
        part = [x[a:a + 5000].contiguous() for x in (q, k)]
        want = binding.qk_norm_rope(*part, *common, pos[a:a + 5000].contiguous(), freq)
        back = binding.qk_norm_rope_backward(*part, *part, *common, pos[a:a + 5000].contiguous(), freq)
        for i in range(2):
            assert torch.equal(out[i][a:a + 5000], want[i]) and torch.equal(grads[i][a:a + 5000], back[i])
    del q, k, out, grads
    torch.cuda.empty_cache()


def test_repeats_streams_and_graphs():
    import torch
    cases = [Case(7 + i, 700 + i, 6, 2, 64, 64) for i in range(2)]
    step = lambda c: (*run(c), *run_backward(c))  # noqa: E731
    want = [step(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
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
            c.q.add_(0.5)
        fresh = [step(c) for c in cases]
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip(fresh, held):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), turn
