"""qk_norm_rope by positions of several axes on views of one projection's
output, as a model passes them: 16-byte aligned ones, whose lanes take four
pairs, and ones at odd multiples of 4 bytes, whose lanes take one.  Everything
around inputs is NaN, everything around results is kept."""
import pytest

from _gpu import device, say
from test_rope_axes import Case, check, run, run_backward

pytestmark = pytest.mark.gpu

SENTINEL = -777.0
# head widths on both sides of each number of lanes, rotated in whole and in part
HEADS = [(32, 32), (64, 64), (64, 48), (96, 48), (128, 128), (128, 32), (130, 66), (256, 256)]


def views(arrays, pad, fill):
    """Copies of two [T, heads, d] tensors as columns of one buffer with `pad` columns on either side, and the buffer."""
    import torch
    T, d = arrays[0].shape[0], arrays[0].shape[2]
    wide = [a.shape[1] * d for a in arrays]
    buf = torch.full((T + 2, 2 * pad + sum(wide)), fill, device=device())
    parts = buf[1:-1, pad:pad + sum(wide)].split(wide, 1)
    for p, a in zip(parts, arrays):
        p.copy_(a.flatten(1))
    return [p.unflatten(1, (-1, d)) for p in parts], buf


def kept(buf, pad):
    return bool((buf[[0, -1]] == SENTINEL).all()) and bool((buf[:, :pad] == SENTINEL).all()) \
        and bool((buf[:, -pad:] == SENTINEL).all())


def shifted(t):
    """A dense copy that starts 4 bytes behind a 16-byte boundary."""
    import torch
    buf = torch.empty(t.numel() + 1, device=device())
    buf[1:].copy_(t.flatten())
    return buf[1:].view(t.shape)


@pytest.mark.parametrize("d,rotated", HEADS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pad", [4, 1])
def test_views(d, rotated, interleaved, pad):
    """The bits of dense tensors of the same alignment, which the oracle bounds."""
    import torch
    c = Case(d + pad, 75, 5, 2, d, rotated, turns=True, interleaved=interleaved, wide=interleaved)
    if pad == 1:
        c.q, c.k, c.gq, c.gk = (shifted(t) for t in (c.q, c.k, c.gq, c.gk))
    check(c, f"axes views d {d} rotated {rotated} pad {pad}")
    want, grads = run(c), run_backward(c)
    (c.q, c.k), _ = views((c.q, c.k), pad, float("nan"))
    (c.gq, c.gk), _ = views((c.gq, c.gk), pad, float("nan"))
    got, got_grads = run(c), run_backward(c)
    assert all(torch.equal(a, b) for a, b in zip((*got, *got_grads), (*want, *grads)))
    (oq, ok), buf = views(want, pad, SENTINEL)
    oq.zero_(), ok.zero_()
    run(c, q_out=oq, k_out=ok)
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1]) and kept(buf, pad)
    (dq, dk), buf = views(grads[:2], pad, SENTINEL)
    dq.zero_(), dk.zero_()
    run_backward(c, dq=dq, dk=dk)
    assert torch.equal(dq, grads[0]) and torch.equal(dk, grads[1]) and kept(buf, pad)
    # over the gradients and then over the inputs, inside their buffers
    (gq, gk), buf = views((c.gq, c.gk), pad, SENTINEL)
    keep, c.gq, c.gk = (c.gq, c.gk), gq, gk
    again = run_backward(c, dq=gq, dk=gk)
    assert all(torch.equal(a, b) for a, b in zip(again, grads)) and kept(buf, pad)
    c.gq, c.gk = keep
    (c.q, c.k), buf = views((c.q, c.k), pad, SENTINEL)
    run(c, q_out=c.q, k_out=c.k)
    assert torch.equal(c.q, want[0]) and torch.equal(c.k, want[1]) and kept(buf, pad)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", [0, 1])
def test_weights_of_any_alignment(d, which):
    """A weight at an odd multiple of 4 bytes, beside aligned heads."""
    c = Case(which, 75, 5, 2, d, d, turns=True)
    common = list(c.common)
    common[which] = shifted(common[which])
    c.common = tuple(common)
    check(c, f"axes weight {which} d {d}")


@pytest.mark.parametrize("T,hq,hk", [(1, 40, 8), (3, 1, 1), (700, 12, 12)])
def test_few_and_many_tokens(T, hq, hk):
    """A token's heads split over waves, and many tokens, one pair a lane."""
    import torch
    c = Case(T, T, hq, hk, 128, 128, axes=4)
    c.q, c.k, c.gq, c.gk = (shifted(t) for t in (c.q, c.k, c.gq, c.gk))
    check(c, f"axes one pair a lane T {T} heads {hq}/{hk}")
    want = (*run(c), *run_backward(c))
    again = (*run(c), *run_backward(c))
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    say("  the same bits again")
