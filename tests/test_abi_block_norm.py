"""The C boundary of the norms around a block, on the CPU: the argument
structs have the layout that the binding packs, every declared function is
exported, and bad arguments are refused synchronously with the documented
status (fake host addresses; nothing reaches a device)."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, DTYPE, ALIAS, WORKSPACE = 0, -1, -2, -3, -4, -5, -8
BASE, STEP = 0x10000000, 0x1000000


@pytest.fixture(scope="module")
def binding():
    from tiled_dense_gemm_matmul_amd import binding
    return binding


def test_exports(binding):
    lib = binding.load_library()
    with open(os.path.join(ROOT, "include", "block_norm.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = re.findall(r"\b(block_norm[a-z_]*)\s*\(", text)
    assert len(names) == 3
    for fn in names:
        assert hasattr(lib, fn) and fn in binding.EXPORTED, fn


def test_struct_sizes(binding, tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "block_norm.h"\nint main(void) {\nprintf("%zu %zu %zu", '
                   'sizeof(block_norm_problem), sizeof(block_norm_args), sizeof(block_norm_backward_args));\n'
                   'return 0; }\n')
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    sizes = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert sizes == [binding._BLOCK_PROBLEM.size, binding._BLOCK_ARGS.size, binding._BLOCK_BACKWARD_ARGS.size]


PROBLEM = {"pre": BASE, "post": BASE + 0x10000, "gate": BASE + 0x20000, "by_seq": 1, "gate_st": 64, "cu": BASE + 0x30000, "nseq": 3,
           "tokens": 50, "width": 64, "a": 1.0, "b": 1.0, "eps": 1e-6}


def _matrices(*names):
    return {f"{n}{f}": v for i, n in enumerate(names, 1) for f, v in (("", BASE + i * STEP), ("_st", 64))}


FORWARD = {**PROBLEM, **_matrices("x", "y", "x_out", "h")}
BACKWARD = {**PROBLEM, **_matrices("dx_out", "dh", "x_out", "y", "dx", "dy"), "dpre": BASE + 0x40000,
            "dpost": BASE + 0x50000, "dgate": BASE + 0x60000, "dgate_st": 64, "ws": BASE + 9 * STEP, "wsb": 1 << 20}


def forward(binding, **kw):
    assert not set(kw) - set(FORWARD)
    return binding.load_library().block_norm(binding._BLOCK_ARGS.pack(*{**FORWARD, **kw}.values()), None)


def backward(binding, **kw):
    assert not set(kw) - set(BACKWARD)
    return binding.load_library().block_norm_backward(
        binding._BLOCK_BACKWARD_ARGS.pack(*{**BACKWARD, **kw}.values()), None)


def workspace(binding, **kw):
    p = {**PROBLEM, **kw}
    return binding.load_library().block_norm_backward_workspace_bytes(binding._BLOCK_PROBLEM.pack(*p.values()))


BAD_PROBLEMS = [({"tokens": -1}, SHAPE), ({"tokens": 1 << 30}, SHAPE), ({"width": 0}, SHAPE), ({"width": 8193}, SHAPE),
                ({"width": -4}, SHAPE), ({"nseq": -1}, SHAPE), ({"nseq": 1 << 24}, SHAPE), ({"by_seq": 2}, DTYPE),
                ({"a": float("nan")}, DTYPE), ({"a": 1e300}, DTYPE), ({"b": float("inf")}, DTYPE), ({"eps": -1e-9}, DTYPE),
                ({"eps": float("nan")}, DTYPE), ({"eps": 1e39}, DTYPE), ({"cu": 0}, NULL), ({"gate_st": -1}, SHAPE), ({"gate_st": 1 << 56}, SHAPE),
                ({"pre": BASE + 2}, ALIGN),
                ({"post": BASE + 0x10001}, ALIGN), ({"gate": BASE + 0x20002}, ALIGN), ({"cu": BASE + 0x30001}, ALIGN)]


@pytest.mark.parametrize("kw,status", BAD_PROBLEMS)
def test_both_passes_refuse_a_problem_alike(binding, kw, status):
    assert forward(binding, **kw) == status
    assert backward(binding, **kw) == status
    assert workspace(binding, **kw) == -1


NO_Y = {"y": 0, "post": 0, "gate": 0, "by_seq": 0}


@pytest.mark.parametrize("kw,status", [
    ({"x": 0}, NULL), ({"x_out": 0}, NULL), ({"h": 0}, NULL), ({**NO_Y, "pre": 0, "x_out": 0, "h": 0}, NULL),
    ({"y": 0}, SHAPE), ({**NO_Y, "post": BASE, "x_out": 0}, SHAPE), ({**NO_Y, "gate": BASE, "x_out": 0}, SHAPE),
    ({**NO_Y}, SHAPE), ({"pre": 0}, SHAPE), ({**NO_Y, "x_out": 0, "a": 0.5}, DTYPE),
    ({**NO_Y, "x_out": 0, "b": 0.5}, DTYPE), ({"x_st": -64}, SHAPE), ({"x_st": 1 << 60}, SHAPE),
    ({"x_out_st": 63}, SHAPE), ({"h_st": 0}, SHAPE), ({"x": BASE + STEP + 2}, ALIGN), ({"h": BASE + 4 * STEP + 1}, ALIGN),
    ({"h": BASE + 3 * STEP}, ALIAS), ({"x_out": BASE + STEP, "x_out_st": 65}, ALIAS), ({"x_out": BASE + STEP + 4}, ALIAS),
    ({"h": BASE + 2 * STEP + 256}, ALIAS), ({"pre": BASE + 4 * STEP + 256}, ALIAS), ({"gate": BASE + 3 * STEP}, ALIAS),
    ({"post": BASE + 3 * STEP + 4}, ALIAS), ({"cu": BASE + 4 * STEP + 8}, ALIAS), ({"tokens": 0}, OK),
    ({"tokens": 0, "x": 0, "y": 0, "x_out": 0, "h": 0}, OK)])
def test_forward_refuses(binding, kw, status):
    assert forward(binding, **kw) == status


@pytest.mark.parametrize("kw,status", [
    ({"dx": 0}, NULL), ({"dy": 0}, NULL), ({"dh": 0}, NULL), ({"x_out": 0}, NULL), ({"dpre": 0}, NULL),
    ({"dpost": 0}, NULL), ({"dgate": 0}, NULL), ({"pre": 0, "dpre": 0, "dh": 0, "dx_out": 0}, NULL),
    ({"y": 0}, SHAPE), ({"pre": 0, "dpre": 0}, SHAPE), ({"pre": 0, "dh": 0}, SHAPE), ({"post": 0}, SHAPE),
    ({"gate": 0}, SHAPE), ({**NO_Y, "dpost": 0, "dgate": 0}, SHAPE),
    ({**NO_Y, "dpost": 0, "dgate": 0, "dy": 0, "b": 2.0}, DTYPE), ({"dx_st": 10}, SHAPE), ({"dgate_st": 63}, SHAPE), ({"dgate_st": 1 << 55}, SHAPE),
    ({"dgate_st": STEP // 4}, ALIAS), ({"dy_st": 0}, SHAPE),
    ({"dh_st": -1}, SHAPE), ({"dx": BASE + 5 * STEP + 2}, ALIGN), ({"dpre": BASE + 0x40001}, ALIGN),
    ({"dgate": BASE + 0x60002}, ALIGN), ({"ws": 0}, WORKSPACE), ({"wsb": 100}, WORKSPACE),
    ({"ws": BASE + 9 * STEP + 8}, ALIGN), ({"dy": BASE + 5 * STEP}, ALIAS), ({"dx": BASE + STEP + 256}, ALIAS),
    ({"dy": BASE + 2 * STEP, "dy_st": 65}, ALIAS), ({"dpre": BASE}, ALIAS), ({"dpost": BASE + 0x40000}, ALIAS),
    ({"dgate": BASE + 0x20000}, ALIAS), ({"dgate": BASE + 0x30000}, ALIAS), ({"dgate": BASE + 4 * STEP + 100}, ALIAS),
    ({"ws": BASE + 3 * STEP}, ALIAS), ({"ws": BASE}, ALIAS), ({"dpre": BASE + 9 * STEP + 16}, ALIAS),
    ({"cu": BASE + 5 * STEP}, ALIAS)])
def test_backward_refuses(binding, kw, status):
    assert backward(binding, **kw) == status


def test_workspace_bytes(binding):
    """One part of each sum a workgroup, and one more of the gate's for every sequence."""
    groups = 13  # 50 rows, 4 a workgroup
    assert workspace(binding) == (3 * groups + 3) * 64 * 4
    assert workspace(binding, gate=0) == 2 * groups * 64 * 4
    assert workspace(binding, by_seq=0) == 3 * groups * 64 * 4
    assert workspace(binding, pre=0, post=0, gate=0) == 0
    assert workspace(binding, width=65, gate=0) == 2 * groups * 68 * 4
    assert workspace(binding, tokens=0, gate=0) == 0
    # short sums stay short: 64 rows a lane at most
    assert workspace(binding, tokens=1 << 20, gate=0, post=0) == (1 << 12) * 64 * 4
    assert binding.load_library().block_norm_backward_workspace_bytes(None) == -1


def test_null_arguments(binding):
    lib = binding.load_library()
    assert lib.block_norm(None, None) == NULL and lib.block_norm_backward(None, None) == NULL
