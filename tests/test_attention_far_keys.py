"""Attention whose bias pushes far keys out of sight: slopes times distances
from 2^30 to past fp32's range, where a row's own key, which has no bias,
holds all of the probability.  Every way of dealing out rows, forward and
backward; slopes that are no numbers still show."""
import numpy as np
import pytest

from oracle import attention as OA

from _gpu import device, say, to_dev

pytestmark = pytest.mark.gpu

# few rows and many (joined waves, one block and two), and many short
# sequences (each wave its own rows)
PLANS = {"few": dict(lengths=[2000], heads=2), "many": dict(lengths=[2000], heads=64),
         "short": dict(lengths=[250] * 8, heads=64), "tiny": dict(lengths=[40], heads=2),
         "long": dict(lengths=[40000], heads=2)}


def problem(lengths, heads, d, slopes, seed=0, kv=None):
    import torch
    g = torch.Generator(device=device())
    g.manual_seed(seed)
    T = sum(lengths)
    q, do = (torch.randn((T, heads, d), generator=g, device=device()) for _ in range(2))
    k, v = (torch.randn((T, kv or heads, d), generator=g, device=device()) for _ in range(2))
    cu = None if len(lengths) == 1 else to_dev(np.cumsum([0, *lengths]).astype(np.int32))
    return q, k, v, do, {"cu_seqlens": cu, "slopes": torch.full((heads,), slopes, device=device())}


CASES = [(plan, slope, causal, d)
         for plan, slope in (("tiny", 1e10), ("few", 1e7), ("few", 1e38), ("many", 1e7), ("many", 1e30), ("short", 1e8),
                             ("short", 1e38))
         for causal in (True, False) for d in (32, 64, 128)] + [("long", 1e5, True, 64)]


@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("plan,slope,causal,d", CASES)
def test_a_row_is_left_its_own_key(plan, slope, causal, d, softcap):
    """The nearest other key is 1e5 or more below a row's own, so that one's
    probability is 1 but for the rounding of the exponent that is taken back
    out of lse: out is v to two roundings (the sum's reciprocal and the
    product), lse the score as the single key's of test_attention_scores.py,
    and dv within 2^-22 of dout.  What other keys would add is exp(-1e5) = 0,
    so the slopes' gradient, whose only term is at distance 0, is zero."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    q, k, v, do, kw = problem(d=d, slopes=slope, **PLANS[plan])
    kw.update(causal=causal, softcap=softcap)
    out, lse = binding.attention(q, k, v, **kw)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    assert bool(((out - v).abs() <= 3 * 2.0 ** -24 * v.abs()).all())
    score = (q.double() * k.double()).sum(2) / d ** 0.5
    size = (q.double() * k.double()).abs().sum(2) / d ** 0.5
    if softcap:
        score = softcap * torch.tanh(score / softcap)
    # d products and the scale, the cap's 8 u, lse's own 2^-23 and rounding
    bound = ((d + 6) * size + 10 * score.abs() + 4) * 2.0 ** -24
    assert bool(((lse.t().double() - score).abs() <= bound).all())
    ds = torch.full_like(kw["slopes"], 9.0)
    dq, dk, dv, _ = binding.attention_backward(do, q, k, v, out, lse, dslopes=ds, **kw)
    assert bool(torch.isfinite(dq).all()) and bool(torch.isfinite(dk).all()) and not ds.any()
    assert bool(((dv - do).abs() <= 2.0 ** -22 * do.abs()).all())


@pytest.mark.parametrize("slope", [1e10, 3e7, 1e38])
@pytest.mark.parametrize("heads,kv,prefix", [(2, 1, None), (6, 2, 25), (128, 128, 40)])
def test_against_the_oracle(slope, heads, kv, prefix):
    """One head's far keys out of sight, its neighbours' as near as ever."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    lengths = [100, 33, 1, 250, 128]
    q, k, v, do, kw = problem(lengths, heads, 32, 0.1, seed=heads, kv=kv)
    kw["slopes"][::2] = slope
    host = {"cu": kw["cu_seqlens"].cpu().numpy(), "slopes": kw["slopes"].cpu().numpy()}
    if prefix is not None:
        host["prefix"] = np.full(5, prefix, np.int32)
        kw["prefix_lens"] = to_dev(host["prefix"])
    out, lse = binding.attention(q, k, v, **kw)
    got = binding.attention_backward(do, q, k, v, out, lse, dslopes=torch.empty_like(kw["slopes"]), **kw)
    q, k, v, do, out, lse = (x.cpu().numpy() for x in (q, k, v, do, out, lse))
    ro, rl, eo, el = OA.scored_attention(q, k, v, **host)
    want = OA.scored_attention_backward(do, q, k, v, out, lse, **host)
    for name, y, ref, err in [("out", out, ro, eo), ("lse", lse, rl, el),
                              *[(n, got[i].cpu().numpy(), want[i], want[4 + i])
                                for i, n in enumerate(("dq", "dk", "dv", "dslopes"))]]:
        res = OA.compare(y, ref, err)
        say(f"  far keys {slope} {heads}/{kv} {name}: max err/bound {res['max_ratio']:.3g}, fails {res['fails']}")
        assert res["fails"] == 0, (name, res)


@pytest.mark.parametrize("plan", ["few", "many", "short"])
def test_no_number_is_hidden(plan):
    """NaN in a query, and slopes that are no finite numbers, reach their rows and heads and no others."""
    import torch
    from tiled_dense_gemm_matmul_amd import binding
    q, k, v, _, kw = problem(d=32, slopes=1e7, **PLANS[plan])
    out, lse = binding.attention(q, k, v, **kw)
    q[77, 0] = float("nan")
    got, got_lse = binding.attention(q, k, v, **kw)
    assert bool(got[77, 0].isnan().all()) and bool(got_lse[0, 77].isnan())
    keep = torch.ones_like(out[:, :, 0], dtype=torch.bool)
    keep[64:96, 0] = False  # of the same block of rows
    assert torch.equal(got[keep], out[keep]) and torch.equal(got_lse.t()[keep], lse.t()[keep])
    q[77, 0] = 0.0
    for bad in (float("nan"), float("inf"), -float("inf")):
        kw["slopes"][1] = bad
        got, got_lse = binding.attention(q, k, v, **kw)
        assert bool(got[:, 1].isnan().all()) and bool(got_lse[1].isnan().all())
        assert bool(torch.isfinite(got[:, 0]).all())
