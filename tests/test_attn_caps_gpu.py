"""GPU tests of capped scores over caps of every size.

Queries and keys are small whole numbers and the scale is a power of two, so that
the scores are exact before they are capped. Bounds, with X the largest capped
score of the batch and u as in attn_cases.py: a capped score is off by
e = 2^-20 X + 2^-22 at most (a factor into the cap, the tanh within 2^-21 of
itself, a factor out of it, log2 units and the softmax's subtraction: roundings of
2^-24 each, below 2^-20 together), and 2^-22 of the cap where it is 64 or less (the
tanh within 2^-22 absolute); results by u |ref| + (u + 2 e) A + 2^-24, as
a numerator over the sum changes by exp(2 e); the logarithm of the sum by e and
its own rounding, 1e-5 + 2^-22 |ref|."""
import math

import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn_cases as ac

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16


def _run(lens, hq, hk, d, page, dtype, softcap, ratio, most=3, seed=3, **kw):
    """One batch of whole numbers up to `most` whose largest score is `ratio` of the
    cap, about."""
    g = torch.Generator().manual_seed(seed)
    n, kv = [a for a, _ in lens], [b for _, b in lens]
    q = torch.randint(-most, most + 1, (sum(n), hq, d), generator=g).to(dtype)
    used = [-(-b // page) for b in kv]
    kp = torch.randint(-most, most + 1, (sum(used), hk, page, d), generator=g).to(dtype)
    vp = torch.randn(sum(used), hk, page, d, generator=g).to(dtype)
    # products of d values have this spread; the largest are some 4.5 times as much
    spread = most * (most + 1) / 3 * math.sqrt(d)
    scale = 2.0 ** round(math.log2(softcap) + math.log2(ratio / (4.5 * spread)))
    table = torch.zeros(len(lens), max(used), dtype=torch.int32)
    outs, bounds, lses, top, page0, row = [], [], [], 0.0, 0, 0
    for s, (a, b) in enumerate(lens):
        table[s, :used[s]] = torch.arange(page0, page0 + used[s])
        flat = [t[page0:page0 + used[s]].transpose(1, 2).reshape(-1, hk, d)[:b] for t in (kp, vp)]
        o, bound, l = ac.sequence(q[row:row + a], *flat, scale, softcap, **kw)
        outs.append(o), bounds.append(bound), lses.append(l)
        x = torch.einsum("nhd,jhd->hnj", q[row:row + a].double(),
                         flat[0].double().repeat_interleave(hq // hk, dim=1)) * scale
        top = max(top, float((softcap * torch.tanh(x / softcap)).abs().max()))
        page0 += used[s]
        row += a
    layer = moe.PagedAttention(hq, hk, d, page, sum(n), len(lens), dtype=dtype)
    cu = torch.tensor([0] + n).cumsum(0).to(torch.int32)
    out, lse = layer.forward(q.to(DEV), kp.to(DEV), vp.to(DEV), table.to(DEV), cu.to(DEV),
                             torch.tensor(kv, dtype=torch.int32, device=DEV), max(n),
                             scale=scale, softcap=softcap, return_lse=True, **kw)
    want, a, want_lse = torch.cat(outs), torch.cat(bounds), torch.cat(lses)
    e, u = 2.0 ** -20 * top + 2.0 ** -22, ac.ROUND[dtype]
    if softcap <= 64.0:
        e += 2.0 ** -22 * softcap
    gap = (lse.cpu().double() - want_lse).abs()
    assert bool((gap <= e + 1e-5 + 2.0 ** -22 * want_lse.abs()).all()), (float(gap.max()), e)
    err = (out.cpu().double() - want).abs()
    # (where 2 e is not small, exp(2 e) - 1 takes its place, up to the whole of A)
    assert bool((err <= u * want.abs() + (u + min(2.0, math.expm1(2 * e))) * a
                 + 2.0 ** -24).all()), float(err.max())
    assert layer.check_device_errors() == 0


@pytest.mark.parametrize("softcap", [0.01, 30.0, 1e3, 2e3, 1e4, 1e5])
@pytest.mark.parametrize("d,dtype,most", [(128, BF, 128), (64, FP, 128), (128, FP, 3)])
def test_whole_blocks_below_the_cap(softcap, d, dtype, most):
    # prompts whose keys fill their blocks, scores up to half of the cap, from
    # products as large as 250000 (scale / cap of 2e-6) and as small as 200
    _run([(40, 384), (200, 256)], 8, 2, d, 64, dtype, softcap, 0.5, most)


@pytest.mark.parametrize("softcap,ratio", [
    (30.0, 0.02), (30.0, 0.6), (30.0, 4.0), (1e3, 0.01), (1e5, 1e-3), (1e5, 0.9), (1e8, 1e-6),
    (1e8, 2.0), (3.4e38, 1e-37), (1e-3, 3.0), (1e-30, 1e6)])
@pytest.mark.parametrize("hq,hk,d,page,dtype", [(8, 2, 128, 16, BF), (4, 4, 64, 64, FP)])
@pytest.mark.parametrize("lens", [
    [(40, 300), (1, 5), (150, 150), (3, 700)],   # the last blocks are in part empty
    [(1, 300), (1, 5), (2, 129), (4, 700), (1, 64)],
])
def test_scores_of_any_size(softcap, ratio, hq, hk, d, page, dtype, lens):
    _run(lens, hq, hk, d, page, dtype, softcap, ratio)


def test_a_large_cap_is_no_cap():
    # standard normal values, scores below 10: a cap of 10^6 moves them by less than 10^-9
    for lens in ([(40, 300), (200, 1000)], [(1, 300), (4, 2000)]):
        for d in (64, 128):
            b = ac.Batch(lens, 8, 2, d, 32, BF)
            layer = moe.PagedAttention(8, 2, d, 32, b.tokens, 2)
            for softcap in (1e6, 1e9, 3.4e38):
                b.check(*b.run(layer, softcap=softcap))


def test_a_row_of_nan_stays_alone():
    for lens in ([(40, 300)], [(4, 300)]):
        b = ac.Batch(lens, 8, 2, 64, 32, BF, softcap=20.0)
        layer = moe.PagedAttention(8, 2, 64, 32, b.tokens, 1)
        b.q[2, 3] = math.nan
        out, lse = b.run(layer)
        assert bool(out[2, 3].isnan().all()) and bool(lse[2, 3].isnan())
        out[2, 3], lse[2, 3] = b.want[2, 3].to(out), b.want_lse[2, 3].to(lse)
        b.check(out, lse)
