"""The block norm's kernels in the built library are those that a width from 1
to 8192 takes: lanes of a row as few as hold it at 16 values each, in groups
of 4, and whole groups or a last one of 1 to 3 values."""
import re


def test_every_kernel_has_its_widths():
    from tiled_dense_gemm_matmul_amd import binding
    taken = set()
    for width in range(1, 8193):
        lanes = 64 if width <= 1024 else 256 if width <= 4096 else 512
        taken.add((lanes, -(-width // (4 * lanes)), width % 4 == 0))
    with open(binding.library_path(), "rb") as f:
        names = re.findall(rb"block_norm_(fwd|bwd)ILi(\d+)ELi(\d+)ELb([01])E", f.read())
    for which in (b"fwd", b"bwd"):
        built = {(int(lanes), int(groups), whole == b"1") for name, lanes, groups, whole in names if name == which}
        assert built == taken
