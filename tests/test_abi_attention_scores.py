"""The C boundary of capped, biased and prefix-masked attention, on the CPU:
argument structs, exports, and bad arguments refused synchronously with the
documented status (fake host addresses; nothing reaches a device)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, DTYPE, ALIAS, WORKSPACE = 0, -1, -2, -3, -4, -5, -8
BASE, STEP = 0x10000000, 0x1000000


@pytest.fixture(scope="module")
def binding():
    from tiled_dense_gemm_matmul_amd import binding
    return binding


def test_struct_sizes(binding, tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "attention.h"\nint main(void) {\nprintf("%zu %zu", '
                   'sizeof(attn_scored_forward_args), sizeof(attn_scored_backward_args));\nreturn 0; }\n')
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    sizes = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert sizes == [binding._SCORED_ARGS.size, binding._SCORED_BACKWARD_ARGS.size]


PROBLEM = {"cu": BASE, "nseq": 3, "tokens": 100, "hq": 4, "hk": 2, "d": 64, "causal": 1, "window": 0, "scale": 0.125}
SCORES = {"softcap": 30.0, "slopes": BASE + 0x10000, "prefix": BASE + 0x20000}


def _tensors(**heads):
    out = {}
    for i, (n, h) in enumerate(heads.items(), 1):
        out.update({n: BASE + i * STEP, n + "_st": h * 64, n + "_sh": 64})
    return out


FORWARD = {**PROBLEM, **SCORES, **_tensors(q=4, k=2, v=2, o=4), "lse": BASE + 0x30000}
BACKWARD = {**PROBLEM, **SCORES, **_tensors(g=4, q=4, k=2, v=2, o=4), "lse": BASE + 0x30000}
BACKWARD.update({n + f: v for i, (n, h) in enumerate((("dq", 4), ("dk", 2), ("dv", 2)), 6)
                 for f, v in (("", BASE + i * STEP), ("_st", h * 64), ("_sh", 64))})
BACKWARD.update({"dslopes": BASE + 0x40000, "ws": BASE + 9 * STEP, "wsb": 1 << 20})


def forward(binding, **kw):
    assert not set(kw) - set(FORWARD)
    return binding.load_library().attn_scored_forward(binding._SCORED_ARGS.pack(*{**FORWARD, **kw}.values()), None)


def backward(binding, **kw):
    assert not set(kw) - set(BACKWARD)
    return binding.load_library().attn_scored_backward(
        binding._SCORED_BACKWARD_ARGS.pack(*{**BACKWARD, **kw}.values()), None)


@pytest.mark.parametrize("kw,status", [
    ({"softcap": -1.0}, DTYPE), ({"softcap": 1e-7}, DTYPE), ({"softcap": 2e6}, DTYPE), ({"softcap": float("nan")}, DTYPE),
    ({"softcap": float("inf")}, DTYPE), ({"softcap": 1e6, "scale": 1e-35}, DTYPE),
    ({"softcap": 1e-6, "scale": 1e35}, DTYPE), ({"causal": 0}, DTYPE), ({"slopes": BASE + 0x10002}, ALIGN),
    ({"prefix": BASE + 0x20001}, ALIGN), ({"d": 66}, SHAPE), ({"tokens": -1}, SHAPE), ({"scale": 0.0}, DTYPE),
    ({"hk": 3}, SHAPE), ({"nseq": -2}, SHAPE), ({"q": 0}, NULL), ({"v": 0}, NULL), ({"lse": 0}, NULL),
    ({"q": BASE + 2 * STEP + 8}, ALIGN)])
def test_both_passes_refuse_alike(binding, kw, status):
    assert forward(binding, **kw) == status and backward(binding, **kw) == status


@pytest.mark.parametrize("kw,status", [
    ({"slopes": BASE + 4 * STEP}, ALIAS), ({"prefix": BASE + 4 * STEP + 64}, ALIAS), ({"cu": BASE + 4 * STEP}, ALIAS),
    ({"slopes": BASE + 0x30000}, ALIAS), ({"prefix": BASE + 0x30004}, ALIAS), ({"o": BASE + 2 * STEP}, ALIAS),
    ({"lse": BASE + STEP}, ALIAS), ({"tokens": 0}, OK)])
def test_forward_refuses(binding, kw, status):
    assert forward(binding, **kw) == status


@pytest.mark.parametrize("kw,status", [
    ({"slopes": 0}, NULL), ({"dslopes": BASE + 0x40001}, ALIGN), ({"dslopes": BASE + 0x10004}, ALIAS),
    ({"dslopes": BASE + 0x20000}, ALIAS), ({"dslopes": BASE + 8}, ALIAS), ({"dslopes": BASE + 0x30008}, ALIAS),
    ({"dslopes": BASE + 6 * STEP}, ALIAS), ({"dslopes": BASE + 3 * STEP + 8}, ALIAS),
    ({"dslopes": BASE + 9 * STEP + 8}, ALIAS), ({"ws": 0}, WORKSPACE), ({"wsb": 40}, WORKSPACE),
    ({"ws": BASE + 9 * STEP + 4}, ALIGN), ({"ws": BASE + 7 * STEP}, ALIAS), ({"ws": BASE + 0x10000 - 64}, ALIAS),
    ({"slopes": BASE + 8 * STEP}, ALIAS), ({"prefix": BASE + 6 * STEP}, ALIAS), ({"dk": BASE + 2 * STEP}, ALIAS)])
def test_backward_refuses(binding, kw, status):
    assert backward(binding, **kw) == status


def test_workspace_bytes(binding):
    """Nothing for few rows without the slopes' gradient; four parts a tile and head with it, behind delta."""
    def ws(slopes, **kw):
        p = {**PROBLEM, **kw}
        return binding.load_library().attn_scored_backward_workspace_bytes(binding._PROBLEM.pack(*p.values()), slopes)
    assert ws(0) == 0 and ws(1) == 4 * (100 // 16 + 3) * 4 * 8
    delta = 4 * 8191 * 4
    assert ws(0, tokens=8191, cu=0) == delta
    assert ws(1, tokens=8191, cu=0) > delta and (ws(1, tokens=8191, cu=0) - delta) % (4 * 4 * 8) in (0, 4, 8)
    assert ws(1, d=66) == -1
    assert binding.load_library().attn_scored_backward_workspace_bytes(None, 1) == -1


def test_null_arguments(binding):
    lib = binding.load_library()
    assert lib.attn_scored_forward(None, None) == NULL and lib.attn_scored_backward(None, None) == NULL


def test_exports(binding):
    for fn in ("attn_scored_forward", "attn_scored_backward", "attn_scored_backward_workspace_bytes",
               "attn_qk_norm_rope_axes", "attn_qk_norm_rope_axes_backward"):
        assert hasattr(binding.load_library(), fn) and fn in binding.EXPORTED
