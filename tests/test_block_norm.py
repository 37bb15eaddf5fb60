"""block_norm and block_norm_backward on the GPU against the oracle
(oracle/block_norm.py): every lane layout, widths that are no multiple of 4,
every combination of norms and gates, packed sequences of no rows to many,
rows of no sequence, strided and misaligned views inside poisoned buffers,
results over the inputs, streams and graph replays, long sums, more sequences
than one look finds.  The bounds are the oracle's, counted per element."""
import numpy as np
import pytest

from oracle import block_norm as OB

from _gpu import device, say, to_dev

pytestmark = pytest.mark.gpu

SENTINEL = -777.0
GRADS = ("dx", "dy", "dpre_weight", "dpost_weight", "dgate")


class Case:
    """Host arrays and their device tensors, each [tokens, width] one a view of
    a buffer with `pad` poisoned columns and a poisoned row on either side."""

    def __init__(self, seed, lengths, width, first=0, tail=0, pre=True, post=True, gate="sequence", a=1.0, b=1.0,
                 pad=0, y=True, dx_out=True, cu=True, gain=1.0):
        r = np.random.default_rng(seed)
        n = lambda *s: (r.standard_normal(s) * gain).astype(np.float32)  # noqa: E731
        self.T, self.W, self.pad = first + sum(lengths) + tail, width, pad
        self.cu = np.cumsum([first] + list(lengths)).astype(np.int32) if cu else None
        self.used = np.zeros(self.T, dtype=bool)
        for s0, s1 in OB.sequences(self.cu, self.T):
            self.used[s0:s1] = True
        weight = lambda *s: (1 + 0.2 * r.standard_normal(s)).astype(np.float32)  # noqa: E731
        self.shared = {"pre_weight": weight(width) if pre else None, "post_weight": weight(width) if post else None,
                       "gate": {"none": None, "shared": weight(width),
                                "sequence": weight(len(lengths), width)}[gate]}
        self.scales = {"residual_scale": a, "block_scale": b}
        self.x, self.g = n(self.T, width), n(self.T, width) if dx_out else None
        self.y = n(self.T, width) if y else None
        self.gh = n(self.T, width) if pre else None
        self.kw = {k: None if v is None else to_dev(v) for k, v in self.shared.items()}
        self.kw.update(self.scales, cu_seqlens=None if self.cu is None else to_dev(self.cu))
        self.dx_, self.dy_, self.dg, self.dgh = (self.view(v) for v in (self.x, self.y, self.g, self.gh))

    def buffer(self, value):
        import torch
        return torch.full((self.T + 2, self.W + 2 * self.pad), value, device=device())

    def inside(self, buf):
        return buf[1:-1, self.pad:self.pad + self.W]

    def view(self, a):
        """A poisoned buffer's view with `a` in the rows of sequences."""
        if a is None:
            return None
        t = self.inside(self.buffer(float("nan")))
        rows = to_dev(np.flatnonzero(self.used))
        t[rows] = to_dev(a[self.used])
        return t

    def forward(self, **kw):
        from tiled_dense_gemm_matmul_amd import binding
        return binding.block_norm(self.dx_, self.dy_, **self.kw, **kw)

    def backward(self, x_out, **kw):
        from tiled_dense_gemm_matmul_amd import binding
        return binding.block_norm_backward(self.dg, self.dgh, x_out, self.dy_, **self.kw, **kw)

    def oracle(self):
        return OB.block_norm(self.x, self.y, **self.shared, **self.scales, cu=self.cu)

    def oracle_backward(self, x_out):
        return OB.block_norm_backward(self.g, self.gh, x_out, self.y, **self.shared, **self.scales, cu=self.cu)


def close(label, name, y, ref, bound):
    res = OB.compare(y.cpu().numpy(), ref, bound)
    say(f"  {label} {name}: max err/bound {res['max_ratio']:.3g}, fails {res['fails']} of {res['n']}")
    assert res["fails"] == 0, (label, name, res)


def check(c, label):
    import torch
    say(label)
    out, h = c.forward()
    torch.cuda.synchronize()
    ro, rh, eo, eh = c.oracle()
    if c.y is not None:
        close(label, "x_out", out, ro, eo)
    else:
        assert out is c.dx_
    assert (h is None) == (rh is None)
    if h is not None:
        close(label, "h", h, rh, eh)
    got = dict(zip(GRADS, c.backward(out)))
    torch.cuda.synchronize()
    want = c.oracle_backward(out.cpu().numpy())
    assert {k for k, v in got.items() if v is not None} == set(want)
    for k, (ref, bound) in want.items():
        close(label, k, got[k], ref, bound)


# on both sides of each bound at which a row gets another group of 4 or more lanes
WIDTHS = [1, 2, 3, 4, 5, 64, 255, 256, 257, 260, 512, 516, 767, 768, 772, 1022, 1024, 1025, 1028, 1150, 2048, 2052, 3070,
          4095, 4096, 4097, 4100, 6144, 6148, 8190, 8192]


@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width):
    check(Case(width, [9, 0, 1, 7], width, first=2, tail=3, a=0.9, b=0.4), f"block_norm width {width}")


@pytest.mark.parametrize("width", [100, 1030, 5000])
@pytest.mark.parametrize("pre,post", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate,cu", [("none", False), ("none", True), ("shared", False), ("shared", True),
                                     ("sequence", True)])
def test_parts(width, pre, post, gate, cu):
    """Every combination of norms and gates, with and without sequences."""
    check(Case(width, [5, 14], width, first=1 if cu else 0, tail=2 if cu else 0, pre=pre, post=post, gate=gate, cu=cu,
               a=1.5, b=-0.3), f"block_norm width {width} pre {pre} post {post} gate {gate} cu {cu}")


@pytest.mark.parametrize("width", [96, 2000])
@pytest.mark.parametrize("cu", [True, False])
@pytest.mark.parametrize("dx_out", [True, False])
def test_the_norm_alone(width, cu, dx_out):
    """Without y: in front of the first block, and behind the last, whose stream nothing else reads."""
    check(Case(width, [6, 11], width, tail=2 if cu else 0, post=False, gate="none", y=False, dx_out=dx_out, cu=cu),
          f"block_norm alone {width} cu {cu} dx_out {dx_out}")


@pytest.mark.parametrize("lengths", [[1], [3], [1] * 70, [0, 4, 0, 0, 9, 0], [513], [2048], [700, 1, 699], [64, 65] * 9])
@pytest.mark.parametrize("gate", ["sequence", "shared"])
def test_lengths(lengths, gate):
    check(Case(len(lengths), lengths, 132, tail=5, gate=gate), f"block_norm lengths {str(lengths)[:30]} {gate}")


@pytest.mark.parametrize("number", [63, 64, 65, 4096, 4097, 9001])
def test_many_sequences(number):
    """On both sides of the numbers at which the search takes another look, runs of empty sequences among them."""
    r = np.random.default_rng(number)
    lengths = r.integers(0, 4, number)
    lengths[10:40] = 0
    lengths[number // 2] = 300
    check(Case(number, [int(n) for n in lengths], 36, first=3, tail=4), f"block_norm {number} sequences")


def test_long_sums():
    """More rows than 64 a lane in 512 workgroups: sums over 150000 rows."""
    check(Case(3, [100001, 49999], 8, tail=7), "block_norm long sums")


@pytest.mark.parametrize("gain", [1e-12, 1e-4, 1e6, 1e12])
def test_magnitudes(gain):
    """Rows far smaller than eps, and large ones."""
    check(Case(4, [12, 3], 300, gain=gain, a=0.7), f"block_norm gain {gain}")


@pytest.mark.parametrize("width,pad", [(768, 4), (768, 1), (101, 3), (1150, 1), (4100, 2), (7001, 5)])
def test_views_and_guards(width, pad):
    """Strided and misaligned views, everything around them NaN or kept."""
    import torch
    c = Case(width, [8, 0, 13], width, first=1, tail=2, pad=pad)
    check(c, f"block_norm views {width}+{pad}")
    want = c.forward()
    grads = c.backward(want[0])
    bufs = [c.buffer(SENTINEL) for _ in range(4)]
    views = [c.inside(b) for b in bufs]
    sums = {k: torch.full((v.numel() + 8,), SENTINEL, device=device()) for k, v in zip(GRADS[2:], grads[2:])}
    out = c.forward(x_out=views[0], h_out=views[1])
    assert out[0] is views[0] and out[1] is views[1]
    got = c.backward(want[0], dx=views[2], dy=views[3],
                     **{k: sums[k][4:-4].view(v.shape) for k, v in zip(GRADS[2:], grads[2:])})
    torch.cuda.synchronize()
    for a, b in zip((*want, *grads), (*out, *got)):
        assert torch.equal(a, b)
    for b, v in zip(bufs, views):
        v.fill_(SENTINEL)
        assert bool((b == SENTINEL).all())
    for s in sums.values():
        assert bool((s[:4] == SENTINEL).all()) and bool((s[-4:] == SENTINEL).all())


@pytest.mark.parametrize("width", [768, 1150, 5002])
def test_results_over_inputs(width):
    """x_out and h over x and y, dx and dy over any two of the inputs: the same bits."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    c = Case(1, [70, 33], width, tail=2)
    want = c.forward()
    for swap in (False, True):
        x, y = c.dx_.clone(), c.dy_.clone()
        a, b = (y, x) if swap else (x, y)
        got = binding.block_norm(x, y, **c.kw, x_out=a, h_out=b)
        assert got[0] is a and got[1] is b and torch.equal(a, want[0]) and torch.equal(b, want[1])
    grads = c.backward(want[0])
    for i in range(4):
        for j in range(4):
            if i == j:
                continue
            t = [v.clone() for v in (c.dg, c.dgh, want[0], c.dy_)]
            got = binding.block_norm_backward(*t, **c.kw, dx=t[i], dy=t[j])
            assert got[0] is t[i] and got[1] is t[j]
            assert all(torch.equal(p, q) for p, q in zip(got, grads)), (i, j)


def test_broadcast_rows():
    """An input whose rows are one row seen several times."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    x, y, w = (torch.randn(s, device=device()) for s in ((1, 200), (31, 200), (200,)))
    got = binding.block_norm(x.expand(31, 200), y, w)
    want = binding.block_norm(x.expand(31, 200).contiguous(), y, w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = binding.block_norm_backward(x.expand(31, 200), y, got[0], y, w)
    want = binding.block_norm_backward(x.expand(31, 200).contiguous(), y, want[0], y, w)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, want))


def test_nothing_passes_between_rows():
    """A row of NaN or infinities stays in its row, and in the sums of its sequence."""
    import torch
    c = Case(2, [40, 30], 260)
    want = c.forward()
    grads = c.backward(want[0])
    for bad in (float("nan"), float("inf")):
        c.dx_[7], c.dy_[7] = bad, bad
        out, h = c.forward()
        got = c.backward(out)
        keep = torch.arange(70, device=device()) != 7
        for a, b in zip((*want, *grads[:2]), (out, h, *got[:2])):
            assert torch.equal(a[keep], b[keep])
        assert torch.equal(grads[4][1], got[4][1]) and bool(got[4][0].isnan().any())


def test_no_rows():
    """No tokens, no sequence, and sequences of none: zero sums."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    dev = device()
    w = torch.ones(20, device=dev)
    e = torch.empty((0, 20), device=dev)
    gate, cu = torch.ones((2, 20), device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    out, h = binding.block_norm(e, e, w, w, gate, cu_seqlens=cu)
    assert out.shape == h.shape == (0, 20)
    dx, dy, *sums = binding.block_norm_backward(e, e, e, e, w, w, gate, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert dx.shape == dy.shape == (0, 20) and all(not s.any() for s in sums) and sums[2].shape == (2, 20)
    x = torch.full((9, 20), float("nan"), device=dev)
    for cu, gate in ((cu, gate), (cu[:1], gate[:0])):
        out, h = binding.block_norm(x, x, w, w, gate, cu_seqlens=cu)
        dx, dy, *sums = binding.block_norm_backward(x, x, x, x, w, w, gate, cu_seqlens=cu)
        torch.cuda.synchronize()
        assert not any(bool(t.any()) for t in (out, h, dx, dy, *sums))


def test_bounds_of_sequences_are_clamped():
    import torch
    c = Case(5, [20, 30], 100, tail=0)
    want = c.forward()
    grads = c.backward(want[0])
    c.kw["cu_seqlens"] = torch.tensor([-9, 20, 1000], dtype=torch.int32, device=device())
    got = c.forward()
    assert all(torch.equal(a, b) for a, b in zip((*want, *grads), (*got, *c.backward(got[0]))))


def test_bounds_that_decrease_stay_inside():
    """Any entries: the rows outside the call's arrays are kept (the results are unspecified)."""
    import torch
    c = Case(5, [20, 30, 10, 40], 100, tail=3)
    r = np.random.default_rng(1)
    for _ in range(20):
        c.kw["cu_seqlens"] = to_dev(r.integers(-5, 110, 5).astype(np.int32))
        bufs = [c.buffer(SENTINEL) for _ in range(4)]
        views = [c.inside(b) for b in bufs]
        c.forward(x_out=views[0], h_out=views[1])
        c.backward(c.dx_, dx=views[2], dy=views[3])
        torch.cuda.synchronize()
        for b, v in zip(bufs, views):
            assert bool((b[0] == SENTINEL).all()) and bool((b[-1] == SENTINEL).all())


def test_offsets_past_32_bits():
    """Rows 2^14 values apart, past 8 GiB into the buffer."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    T, W = 140000, 40
    g = torch.Generator(device=device())
    g.manual_seed(1)
    buf = torch.empty((T, 16384), device=device())
    buf[:, 64:64 + 2 * W] = torch.randn((T, 2 * W), generator=g, device=device())
    x, y = buf[:, 64:64 + W], buf[:, 64 + W:64 + 2 * W]
    w = torch.randn(W, generator=g, device=device())
    got = binding.block_norm(x, y, w, w, w)
    want = binding.block_norm(x.contiguous(), y.contiguous(), w, w, w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = buf[:, 256:256 + 2 * W]
    a = binding.block_norm_backward(x, y, x, y, w, w, w, dx=out[:, :W], dy=out[:, W:])
    x, y = x.contiguous(), y.contiguous()
    b = binding.block_norm_backward(x, y, x, y, w, w, w)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    del buf, a, b, got, want
    torch.cuda.empty_cache()


def test_gates_as_columns_of_a_projection():
    """Each sequence's gate and its gradient as columns of a wider buffer, and one gate seen by all sequences."""
    import torch
    c = Case(8, [30, 0, 41], 96, tail=3)
    want = c.forward()
    grads = c.backward(want[0])
    wide = torch.full((3, 300), float("nan"), device=device())
    wide[:, 101:197] = c.kw["gate"]
    kept = torch.full((3, 300), SENTINEL, device=device())
    c.kw["gate"] = wide[:, 101:197]
    got = c.forward()
    back = c.backward(got[0], dgate=kept[:, 7:103])
    assert all(torch.equal(a, b) for a, b in zip((*want, *grads), (*got, *back)))
    kept[:, 7:103] = SENTINEL
    assert bool((kept == SENTINEL).all())
    c.kw["gate"] = wide[:1, 101:197].expand(3, 96)
    got = (*c.forward(), *c.backward(want[0]))
    c.kw["gate"] = c.kw["gate"].contiguous()
    assert all(torch.equal(a, b) for a, b in zip(got, (*c.forward(), *c.backward(want[0]))))


def test_more_rows_than_one_launch_takes():
    """40 million rows, a wave each forward: both ends against the same rows alone, and the sums in 64 bits."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    T, W = 40000003, 4
    g = torch.Generator(device=device())
    g.manual_seed(4)
    x, y, gx, gh = (torch.randn((T, W), generator=g, device=device()) for _ in range(4))
    w, gate = torch.randn(W, generator=g, device=device()), torch.randn(W, generator=g, device=device())
    out, h = binding.block_norm(x, y, w, w, gate, 0.9, 0.4)
    dx, dy, *sums = binding.block_norm_backward(gx, gh, out, y, w, w, gate, 0.9, 0.4)
    for rows in (slice(0, 500), slice(33554432 - 250, 33554432 + 250), slice(T - 500, T)):
        part = [t[rows].contiguous() for t in (x, y, gx, gh, out)]
        o2, h2 = binding.block_norm(part[0], part[1], w, w, gate, 0.9, 0.4)
        assert torch.equal(out[rows], o2) and torch.equal(h[rows], h2)
        d2 = binding.block_norm_backward(part[2], part[3], part[4], part[1], w, w, gate, 0.9, 0.4)
        assert torch.equal(dx[rows], d2[0]) and torch.equal(dy[rows], d2[1])
    # dpre: sum of dh out r, in slices of 64 bits; a term is off by some 40 u, its sum in fp32 by 70 more
    total = size = 0.0
    for rows in torch.arange(T, device=device()).split(4000000):
        o = out[rows].double()
        term = gh[rows].double() * o / torch.sqrt((o * o).mean(1, keepdim=True) + 1e-6)
        total, size = total + term.sum(0), size + term.abs().sum(0)
    assert bool(((sums[0].double() - total).abs() <= 120 * 2.0 ** -24 * size).all())
    del x, y, gx, gh, out, h, dx, dy
    torch.cuda.empty_cache()


def test_more_sequences_than_one_launch_takes():
    """Nine million sequences of one row and none: the gate's gradient has a row for each."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    S, W = 9000001, 4
    g = torch.Generator(device=device())
    g.manual_seed(5)
    lengths = torch.randint(0, 2, (S,), generator=g, device=device(), dtype=torch.int32)
    cu = torch.cat((torch.zeros(1, dtype=torch.int32, device=device()), lengths.cumsum(0, dtype=torch.int32)))
    T = int(cu[-1])
    x, y, gx = (torch.randn((T, W), generator=g, device=device()) for _ in range(3))
    gate = torch.randn((S, W), generator=g, device=device())
    seq = torch.repeat_interleave(torch.arange(S, device=device()), lengths.long())
    out, _ = binding.block_norm(x, y, gate=gate, cu_seqlens=cu)
    assert torch.allclose(out, x + gate[seq] * y, rtol=1e-6, atol=1e-6)
    dx, dy, _, _, dgate = binding.block_norm_backward(gx, None, out, y, gate=gate, cu_seqlens=cu)
    assert torch.equal(dx, gx) and torch.equal(dy, gx * gate[seq])
    want = torch.zeros_like(gate)
    want[seq] = gx * y
    assert torch.equal(dgate, want)
    del x, y, gx, gate, out, dx, dy, dgate, want
    torch.cuda.empty_cache()


def test_refusals_on_the_device():
    import torch
    from tiled_dense_gemm_matmul_amd import binding as B
    dev = device()
    x, y, w = torch.randn((9, 64), device=dev), torch.randn((9, 64), device=dev), torch.ones(64, device=dev)
    cu = torch.tensor([0, 4, 9], dtype=torch.int32, device=dev)
    n, b = B.block_norm, B.block_norm_backward
    for bad in (lambda: n(x), lambda: n(x, pre_weight=w, post_weight=w), lambda: n(x, pre_weight=w, gate=w),
                lambda: n(x, pre_weight=w, x_out=y), lambda: n(x, pre_weight=w, residual_scale=2.0),
                lambda: n(x, y, h_out=x), lambda: n(x, y[:8], w), lambda: n(x, y, w[:63]), lambda: n(x, y.cpu(), w),
                lambda: n(x.t().contiguous().t(), y, w), lambda: n(x, y, w, gate=torch.ones((2, 64), device=dev)),
                lambda: n(x, y, w, gate=torch.ones((3, 64), device=dev), cu_seqlens=cu),
                lambda: n(x, y, w, gate=w[:60]), lambda: b(x, None, x, y, w), lambda: b(None, None, x, y),
                lambda: b(x, x, x, y), lambda: b(x, x, x, None, w, dy=y), lambda: b(x, x, x, y, w, dgate=w),
                lambda: b(x, x, x, y, w, gate=w, dgate=w[:60])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: n(x[0], y, w), lambda: n(x.double(), y, w), lambda: n(x, y.half(), w),
                lambda: n(x, y, w, gate=1.0), lambda: n(x, y, w, cu_seqlens=cu.long())):
        with pytest.raises(TypeError):
            bad()
    wide = torch.zeros((2, 8193), device=dev)
    one = torch.randn((1, 64), device=dev)
    for bad, status in ((lambda: n(wide, pre_weight=wide[0]), -2), (lambda: n(x, y, w, eps=-1.0), -4),
                        (lambda: n(x, y, w, block_scale=float("nan")), -4),
                        (lambda: n(x, y, w, residual_scale=1e39), -4), (lambda: n(x, y, w, x_out=x, h_out=x), -5),
                        (lambda: n(x, y, w, x_out=one.expand(9, 64)), -2), (lambda: n(x, y, x[3]), 0),
                        (lambda: n(x, y, x[3], x_out=x), -5), (lambda: n(x[:8], y[:8], w, x_out=x[1:]), -5),
                        (lambda: b(x, x, x, y, w, dx=y, dy=y), -5), (lambda: b(x, x, x, y, w, dpre_weight=w), -5),
                        (lambda: b(x, x, x, y, w, w, dpre_weight=x[0]), -5)):
        if status == 0:
            bad()
            continue
        with pytest.raises(B.GemmError) as e:
            bad()
        assert e.value.status == status


def test_repeated_calls_streams_and_graphs():
    """Calls on two streams at once, and two captured graphs replayed in turn
    with eager calls between, give the eager bits."""
    import torch
    cases = [Case(10 + i, [300, 211 + i, 0, 90], 768 if i else 1150, tail=3) for i in range(2)]

    def step(c):
        out, h = c.forward()
        return (out, h, *c.backward(out))

    want = [step(c) for c in cases]
    for _ in range(2):
        for c, a in zip(cases, want):
            assert all(torch.equal(p, q) for p, q in zip(a, step(c)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):
        got = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(step(c))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    graphs, held = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(step(c))
        graphs.append(g)
    for turn in range(3):
        for c in cases:
            c.dx_.mul_(1.25)
        fresh = [step(c) for c in cases]
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip(fresh, held):
            assert all(torch.equal(p, q) for p, q in zip(a, b)), turn


@pytest.mark.parametrize("width", [768, 1150, 5002])
def test_verification_build(width, monkeypatch):
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    c = Case(width, [300, 0, 77], width, tail=3)
    out, h = c.forward()
    got = (out, h, *c.backward(out))
    monkeypatch.setattr(binding, "_lib", binding.load_sync_check_library())
    want = (*c.forward(), *c.backward(out))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
