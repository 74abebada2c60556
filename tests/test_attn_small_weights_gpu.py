"""GPU tests of softmax weights far below the largest one, which together carry the
result: in fp16 they lie below what the type can hold beside a weight of 1."""
import math

import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn_cases as ac

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,hq,hk", [(1, 2, 1), (3, 4, 4), (40, 4, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("above", [9.0, 14.0, 16.0, 17.5])
@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("seqs", [1, 80])  # cut over many CTAs, and whole in one
def test_one_large_weight_over_many_small_ones(dtype, n, hq, hk, d, above, where, seqs):
    # one key scores `above` more than the others and its value is 0, theirs are 1;
    # all sequences have the same pages
    kv, page = (100000 if seqs == 1 else 20000) + n, 64
    used = -(-kv // page)
    kp = torch.zeros(used, hk, page, d, dtype=dtype, device=DEV)
    vp = torch.ones(used, hk, page, d, dtype=dtype, device=DEV)
    at = 0 if where == "first" else kv - n
    kp[at // page, :, at % page, 3] = above
    vp[at // page, :, at % page] = 0.0
    q = torch.zeros(seqs * n, hq, d, dtype=dtype, device=DEV)
    q[..., 3] = 1.0
    i32 = dict(dtype=torch.int32, device=DEV)
    layer = moe.PagedAttention(hq, hk, d, page, seqs * n, seqs, dtype=dtype)
    for kw in (dict(), dict(slopes=torch.zeros(hq, device=DEV)), dict(prefix=torch.ones(seqs, **i32))):
        out, lse = layer.forward(q, kp, vp, torch.arange(used, **i32).repeat(seqs, 1),
                                 n * torch.arange(seqs + 1, **i32),
                                 torch.full((seqs,), kv, **i32), n, scale=1.0, return_lse=True,
                                 **kw)
        # the largest key lies in front of every query; row i sees kv - n + i others
        others = (kv - n + torch.arange(n, dtype=torch.float64)) * math.exp(-above)
        others = others.repeat(seqs)
        want = (others / (1 + others))[:, None, None].expand(-1, hq, d)
        want_lse = (above + torch.log1p(others))[:, None].expand(-1, hq)
        ac.check_attention(out, lse, want, want, want_lse, dtype)
    assert layer.check_device_errors() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 10, 2.0 ** 18, 2.0 ** 22, 2.0 ** 26, 2.0 ** 40])
@pytest.mark.parametrize("n,hq", [(1, 2), (40, 4)])
@pytest.mark.parametrize("softcap,bias", [(0.0, False), (0.0, True), (3e30, False)])
def test_large_scores_give_the_largest_ones_value(dtype, scale, n, hq, softcap, bias):
    # scores are whole multiples of the scale, exact; where two keys share the largest
    # they share the result. Numerators must not leave the type for any of them, at
    # scores whose fp32 neighbours are 1, 4 or 64 apart
    d, page, kv = 64, 64, 1000 + n
    used = -(-kv // page)
    g = torch.Generator().manual_seed(9)
    kp = torch.randint(-2, 3, (used, 1, page, d), generator=g).to(dtype)
    vp = torch.randn(used, 1, page, d, generator=g).to(dtype)
    q = torch.randint(-2, 3, (n, hq, d), generator=g).to(dtype)
    i32 = dict(dtype=torch.int32, device=DEV)
    layer = moe.PagedAttention(hq, 1, d, page, n, 1, dtype=dtype)
    out, lse = layer.forward(q.to(DEV), kp.to(DEV), vp.to(DEV), torch.arange(used, **i32)[None],
                             torch.tensor([0, n], **i32), torch.tensor([kv], **i32), n,
                             scale=scale, softcap=softcap, return_lse=True,
                             slopes=torch.zeros(hq, device=DEV) if bias else None)
    k, v = (t.transpose(1, 2).reshape(-1, 1, d)[:kv] for t in (kp, vp))
    # (from the largest score down: a logarithm of 10^13 and a sum has no fp64 of its own)
    x = torch.einsum("nhd,jd->hnj", q.double(), k[:, 0].double()) * scale
    x = x.masked_fill(~ac.seen_mask(n, kv), -math.inf)
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - top)
    total = w.sum(-1, keepdim=True)
    want, a = (torch.einsum("hnj,jd->nhd", w / total, y.double()) for y in (v[:, 0], v[:, 0].abs()))
    want_lse = (top + total.log())[..., 0].T
    if softcap:  # a cap far above: a score is off by 2^-21 of itself, ties stay ties
        gap = (lse.cpu().double() - want_lse).abs()
        assert bool((gap <= 1e-4 + 2.0 ** -20 * want_lse.abs()).all())
        lse = None
        if scale < 2.0 ** 10:
            return
    ac.check_attention(out, lse, want, a, want_lse, dtype)
    assert layer.check_device_errors() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("scale", [0.0, 1e-45, 1e-38, 1e-37, 1e-31, 1e-29, -1e-38, -0.2])
@pytest.mark.parametrize("lens", [[(40, 3000), (150, 150)], [(1, 3000), (2, 77)]])
def test_small_and_negative_scales(dtype, scale, lens):
    b = ac.Batch(lens, 8, 2, 64, 32, dtype, scale=scale)
    layer = moe.PagedAttention(8, 2, 64, 32, b.tokens, 2, dtype=dtype)
    b.check(*b.run(layer))
    assert layer.check_device_errors() == 0
