"""qk_norm_rope and its backward pass by positions of several axes: on the CPU
the C boundary's refusals and the oracle's pins, on the GPU every lane layout
of the kernels against the oracle (oracle/attention.py), sections and axes in
turn, far positions, one axis against the plain call bit for bit, entries
outside the axes, results over the inputs, streams and graph replays."""
import os
import subprocess

import numpy as np
import pytest

from oracle import attention as OA

from _gpu import device, say, to_dev

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, DTYPE, ALIAS, WORKSPACE = 0, -1, -2, -3, -4, -5, -8
BASE, STEP = 0x10000000, 0x1000000


@pytest.fixture(scope="module")
def binding():
    from tiled_dense_gemm_matmul_amd import binding
    return binding


# --- on the CPU ---

def test_struct_sizes(binding, tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "attention.h"\nint main(void) {\nprintf("%zu %zu", '
                   'sizeof(attn_qk_norm_rope_axes_args), sizeof(attn_qk_norm_rope_axes_backward_args));\nreturn 0; }\n')
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    sizes = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert sizes == [binding._NORM_AXES_ARGS.size, binding._NORM_AXES_BACKWARD_ARGS.size]


NORM = {"pos": BASE, "pos64": 0, "freq": BASE + 0x10000, "qw": BASE + 0x20000, "kw": BASE + 0x30000, "tokens": 50,
        "hq": 4, "hk": 2, "d": 64, "rotated": 48, "interleaved": 0, "eps": 1e-6, "axis": BASE + 0x40000, "axes": 3}


def _tensors(*names):
    out = {}
    for i, n in enumerate(names, 1):
        heads = 4 if "q" in n else 2
        out.update({n: BASE + i * STEP, n + "_st": heads * 64, n + "_sh": 64})
    return out


FORWARD = {**NORM, **_tensors("q", "k", "q_out", "k_out")}
BACKWARD = {**NORM, **_tensors("dq_out", "dk_out", "q", "k", "dq", "dk"), "dqw": BASE + 0x50000, "dkw": BASE + 0x60000,
            "ws": BASE + 9 * STEP, "wsb": 1 << 22}


def forward(binding, **kw):
    assert not set(kw) - set(FORWARD)
    return binding.load_library().attn_qk_norm_rope_axes(
        binding._NORM_AXES_ARGS.pack(*{**FORWARD, **kw}.values()), None)


def backward(binding, **kw):
    assert not set(kw) - set(BACKWARD)
    return binding.load_library().attn_qk_norm_rope_axes_backward(
        binding._NORM_AXES_BACKWARD_ARGS.pack(*{**BACKWARD, **kw}.values()), None)


@pytest.mark.parametrize("kw,status", [({"axes": 0}, SHAPE), ({"axes": -1}, SHAPE), ({"axes": 65536}, SHAPE),
                                       ({"axis": 0}, NULL), ({"axis": BASE + 2}, ALIGN), ({"pos": 0}, NULL),
                                       ({"tokens": -1}, SHAPE), ({"d": 65}, SHAPE), ({"rotated": 66}, SHAPE),
                                       ({"pos64": 2}, DTYPE), ({"eps": -1.0}, DTYPE), ({"freq": 0}, NULL)])
def test_both_passes_refuse_alike(binding, kw, status):
    assert forward(binding, **kw) == status and backward(binding, **kw) == status


@pytest.mark.parametrize("kw,status", [({"axis": BASE + 3 * STEP}, ALIAS), ({"axis": BASE + 4 * STEP - 48}, ALIAS),
                                       ({"pos": BASE + 4 * STEP - 2 * 50 * 4}, ALIAS), ({"q_out_st": 10}, SHAPE),
                                       ({"k": 0}, NULL), ({"tokens": 0}, OK)])
def test_forward_refuses(binding, kw, status):
    assert forward(binding, **kw) == status


@pytest.mark.parametrize("kw,status", [({"axis": BASE + 5 * STEP}, ALIAS), ({"dqw": BASE + 0x40000}, ALIAS),
                                       ({"axis": BASE + 9 * STEP + 64}, ALIAS), ({"dkw": BASE + 400}, ALIAS),
                                       ({"wsb": 100}, WORKSPACE), ({"dkw": 0}, NULL), ({"dq": BASE + STEP + 4}, ALIAS)])
def test_backward_refuses(binding, kw, status):
    assert backward(binding, **kw) == status


def test_null_arguments(binding):
    lib = binding.load_library()
    assert lib.attn_qk_norm_rope_axes(None, None) == NULL and lib.attn_qk_norm_rope_axes_backward(None, None) == NULL


@pytest.mark.parametrize("interleaved", [True, False])
def test_oracle_of_axes(interleaved):
    """One pair at a time, whose positions are its axis's, and the gradient by differences."""
    r = np.random.default_rng(0)
    T, d, freq, axis = 6, 12, 0.3 ** np.arange(5.0), [2, 0, 1, 1, 0]
    x, w, pos = r.standard_normal((T, 2, d)), r.standard_normal(d), r.integers(0, 50, (3, T))
    y, _ = OA.qk_norm_rope(x, w, pos, freq, interleaved=interleaved, axis=axis)
    for p, a in enumerate(axis):
        whole, _ = OA.qk_norm_rope(x, w, pos[a], freq, interleaved=interleaved)
        cols = [2 * p, 2 * p + 1] if interleaved else [p, p + 5]
        assert np.array_equal(y[..., cols], whole[..., cols])
    dy, step = r.standard_normal(x.shape), r.standard_normal(x.shape)
    dx = OA.qk_norm_rope_backward(dy, x, w, pos, freq, interleaved=interleaved, axis=axis)[0]
    at = lambda e: (OA.qk_norm_rope(x + e * step, w, pos, freq, interleaved=interleaved, axis=axis)[0] * dy).sum()  # noqa: E731
    assert abs((at(1e-5) - at(-1e-5)) / 2e-5 - (dx * step).sum()) < 1e-8
    wrong, bound = OA.qk_norm_rope(x, w, pos, freq, interleaved=interleaved, axis=[2, 0, 1, 0, 0])
    assert OA.compare(wrong, y, bound)["fails"] > 0


def test_oracle_of_far_positions():
    """Against exact fractions, and against the extended product where that is good."""
    from fractions import Fraction
    r = np.random.default_rng(1)
    freq = np.float32([1.0, 0.3, 0.01])
    pos = r.integers(-(1 << 53), 1 << 53, (1, 8))
    angle = OA._angles(pos, freq, [0, 0, 0])
    # 2 pi to 40 digits
    turn = Fraction("6.2831853071795864769252867665590057683943")
    for t, p in enumerate(pos[0]):
        for j, f in enumerate(freq):
            exact = Fraction(int(p)) * Fraction(float(f))
            exact -= round(exact / turn) * turn
            assert abs(float(angle[t, j]) - float(exact)) < 1e-15
    near = r.integers(-(1 << 20), 1 << 20, (1, 8))
    far = np.concatenate([near, np.full((1, 8), 1 << 40)])   # the second row asks for the exact way
    a, b = OA._angles(near, freq, [0, 0, 0]), OA._angles(far, freq, [0, 0, 0])
    assert np.abs(np.exp(1j * a.astype(float)) - np.exp(1j * b.astype(float))).max() < 1e-9


# --- on the GPU ---

class Case:
    def __init__(self, seed, T, hq, hk, d, rotated, axes=3, turns=False, interleaved=False, wide=False, far=1000,
                 gain=1.0):
        r = np.random.default_rng(seed)
        pairs = rotated // 2
        self.x = [(r.standard_normal((T, h, d)) * gain).astype(np.float32) for h in (hq, hk)]
        self.g = [r.standard_normal((T, h, d)).astype(np.float32) for h in (hq, hk)]
        self.w = [(1 + 0.1 * r.standard_normal(d)).astype(np.float32) for _ in range(2)]
        self.pos = r.integers(-far, far, (axes, T)).astype(np.int64 if wide else np.int32)
        self.freq = (10000.0 ** (-np.arange(pairs) / max(1, pairs))).astype(np.float32)
        self.axis = (np.arange(pairs) % axes if turns else np.arange(pairs) * axes // max(1, pairs)).astype(np.int32)
        self.interleaved = interleaved
        self.q, self.k, self.gq, self.gk = (to_dev(a) for a in (*self.x, *self.g))
        self.common = tuple(to_dev(a) for a in (*self.w, self.pos, self.freq))
        self.kw = {"pair_axis": to_dev(self.axis), "interleaved": interleaved}


def run(c, **kw):
    from tiled_dense_gemm_matmul_amd import binding
    return binding.qk_norm_rope(c.q, c.k, *c.common, **c.kw, **kw)


def run_backward(c, **kw):
    from tiled_dense_gemm_matmul_amd import binding
    return binding.qk_norm_rope_backward(c.gq, c.gk, c.q, c.k, *c.common, **c.kw, **kw)


def check(c, label):
    say(label)
    got, grads = run(c), run_backward(c)
    for i, n in enumerate("qk"):
        ref, err = OA.qk_norm_rope(c.x[i], c.w[i], c.pos, c.freq, 1e-6, c.interleaved, c.axis)
        dx, dw, edx, edw = OA.qk_norm_rope_backward(c.g[i], c.x[i], c.w[i], c.pos, c.freq, 1e-6, c.interleaved, c.axis)
        for name, y, r, e in ((n, got[i], ref, err), ("d" + n, grads[i], dx, edx), ("dw", grads[2 + i], dw, edw)):
            res = OA.compare(y.cpu().numpy(), r, e)
            say(f"  {name}: max err/bound {res['max_ratio']:.3g}, fails {res['fails']} of {res['n']}")
            assert res["fails"] == 0, (label, name, res)


@pytest.mark.gpu
@pytest.mark.parametrize("d,rotated", [(2, 2), (8, 8), (16, 8), (32, 32), (64, 48), (96, 96), (128, 64), (130, 66),
                                       (200, 180), (256, 256), (64, 0), (10, 6)])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("turns", [True, False])
def test_layouts(d, rotated, interleaved, turns):
    check(Case(d, 37, 3, 2, d, rotated, turns=turns, interleaved=interleaved, wide=turns), f"axes d {d} rotated {rotated}")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 63, 1025])
@pytest.mark.parametrize("axes", [1, 2, 7])
def test_tokens(T, axes):
    check(Case(T, T, 6, 2, 64, 64, axes=axes, turns=True), f"axes T {T} axes {axes}")


@pytest.mark.gpu
@pytest.mark.parametrize("far", [1 << 20, 1 << 31, 1 << 53])
def test_far_positions(far):
    check(Case(3, 50, 2, 2, 64, 64, far=far, wide=far > 1 << 30), f"axes far {far}")


@pytest.mark.gpu
@pytest.mark.parametrize("d,rotated,interleaved", [(64, 64, False), (96, 48, True), (50, 20, False)])
def test_equal_axes_give_the_plain_bits(d, rotated, interleaved):
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    c = Case(4, 300, 4, 2, d, rotated, turns=True, interleaved=interleaved)
    one = c.common[2][1].contiguous()
    c.common = (*c.common[:2], one.expand(3, 300).contiguous(), c.common[3])
    plain = (*c.common[:2], one, c.common[3])
    want = binding.qk_norm_rope(c.q, c.k, *plain, interleaved=interleaved)
    grads = binding.qk_norm_rope_backward(c.gq, c.gk, c.q, c.k, *plain, interleaved=interleaved)
    assert all(torch.equal(a, b) for a, b in zip((*run(c), *run_backward(c)), (*want, *grads)))


@pytest.mark.gpu
def test_entries_outside_the_axes_are_clamped():
    import torch
    c = Case(5, 40, 2, 1, 32, 32, axes=2)
    c.kw["pair_axis"] = to_dev(np.array([0, 1] * 8, dtype=np.int32))
    want = (*run(c), *run_backward(c))
    c.kw["pair_axis"] = to_dev(np.array([-7, 2000000000] * 8, dtype=np.int32))
    assert all(torch.equal(a, b) for a, b in zip(want, (*run(c), *run_backward(c))))


@pytest.mark.gpu
def test_results_over_inputs_streams_and_graphs():
    import torch
    cases = [Case(6 + i, 200, 4, 2, 64, 64, turns=bool(i)) for i in range(2)]

    def step(c):
        return (*run(c), *run_backward(c))

    want = [step(c) for c in cases]
    for c, w in zip(cases, want):
        q, k, gq, gk = (t.clone() for t in (c.q, c.k, c.gq, c.gk))
        from tiled_dense_gemm_matmul_amd import binding
        binding.qk_norm_rope(q, k, *c.common, **c.kw, q_out=q, k_out=k)
        binding.qk_norm_rope_backward(gq, gk, c.q, c.k, *c.common, **c.kw, dq=gq, dk=gk)
        assert all(torch.equal(a, b) for a, b in zip((q, k, gq, gk), w))
    torch.cuda.synchronize()
    got = []
    for c, s in zip(cases, [torch.cuda.Stream() for _ in cases]):
        with torch.cuda.stream(s):
            got.append(step(c))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(want, got) for a, b in zip(x, y))
    graphs, held = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(step(c))
        graphs.append(g)
    for turn in range(3):
        for c in cases:
            c.q.mul_(1.25)
            c.common[2].add_(1)
        fresh = [step(c) for c in cases]
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(fresh, held) for a, b in zip(x, y)), turn


@pytest.mark.gpu
def test_refusals_on_the_device(binding):
    import torch
    c = Case(8, 20, 2, 1, 32, 32, axes=2)
    w0, w1, pos, freq = c.common
    axis = c.kw["pair_axis"]
    call = lambda pos, axis: binding.qk_norm_rope(c.q, c.k, w0, w1, pos, freq, pair_axis=axis)  # noqa: E731
    for bad in ((pos[0], axis), (pos, None), (pos[:, :19].contiguous(), axis), (pos.t().contiguous().t(), axis),
                (pos, axis[:15]), (pos, axis.cpu()), (pos[None], axis)):
        with pytest.raises(ValueError):
            call(*bad)
    for bad in ((pos, axis.long()), (pos.float(), axis)):
        with pytest.raises(TypeError):
            call(*bad)
    with pytest.raises(binding.GemmError) as e:
        call(pos[:0], axis)
    assert e.value.status in (NULL, SHAPE)
    assert device() == c.q.device and torch.equal(call(pos, axis)[0], run(c)[0])
