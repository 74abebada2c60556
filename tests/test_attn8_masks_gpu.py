"""Rows that see no key, and blocks that no token began, over the 8-bit cache, on each of
its paths."""
import math

import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn8_cases as a8
from tests import attn_cases as ac

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.lib()


def sequence(q, k, v, scale, softcap=0.0, window=0, slopes=None, prefix=0, sinks=0):
    """a8.sequence where rows may stand before the first key, or keys not be there."""
    q, k, v = q.double(), k.double(), v.double()
    n, hq, d = q.shape
    kv, hk = k.shape[0], k.shape[1]
    if kv == 0:
        return (torch.zeros(n, hq, d, dtype=torch.float64),) * 2 + (
            torch.full((n, hq), -math.inf, dtype=torch.float64),)
    head = torch.arange(hq) // (hq // hk)
    x = torch.einsum("nhd,jhd->hnj", q, k[:, head]) * scale
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    p, j = torch.arange(n)[:, None] + (kv - n), torch.arange(kv)[None, :]
    if slopes is not None:
        x = x - slopes.double()[:, None, None] * (p - j).abs()
    near = (j > p - window) | (j < sinks) if window else torch.ones_like(j > p)
    x = x.masked_fill(~(((j <= p) & near) | (j < prefix)), -math.inf)
    lse = torch.logsumexp(x, dim=-1)
    w = torch.exp(x - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[..., None])
    return (torch.einsum("hnj,jhd->nhd", w, v[:, head]),
            torch.einsum("hnj,jhd->nhd", w, v[:, head].abs()), lse.T)


FEW = [(3, 1), (2, 0), (4, 4), (1, 90), (0, 33), (4, 3)]
SOME = [(40, 17), (33, 0), (64, 300), (20, 20), (90, 16), (0, 33), (70, 1)]
MANY = [(200, 130), (190, 0), (300, 300), (160, 1), (150, 700), (0, 12)]


@pytest.mark.parametrize("lens,brought", [(FEW, False), (SOME, False), (MANY, True)])
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, FP)])
@pytest.mark.parametrize("opt", [{}, dict(window=40, sinks=5), dict(softcap=30.0), dict(slopes=True),
                                 dict(prefix=[2, 3, 0, 7, 5, 1, 9])])
def test_rows_that_see_no_key(monkeypatch, lens, brought, d, dtype, opt):
    monkeypatch.setattr(a8, "sequence", sequence)
    opt = dict(opt)
    if "prefix" in opt:
        opt["prefix"] = opt["prefix"][:len(lens)]
    b = a8.Batch8(lens, 8, 2, d, 16, dtype, **opt)
    assert (b.tokens * 4 > 512 * len(lens)) == brought
    empty = int(b.want_lse.isinf().sum())
    assert empty > 0
    layer = moe.PagedAttention(8, 2, d, 16, b.tokens + 3, len(lens), dtype=dtype)
    # rows behind the last sequence stay
    b.q = torch.cat([b.q, b.q[:3]])
    out = torch.full_like(b.q, 5.0)
    lse = torch.full((b.tokens + 3, 8), 5.0, device=DEV)
    for kw in ({}, dict(stream=torch.cuda.current_stream())) if brought else ({},):
        b.run(layer, out=out, lse=lse, **kw)
        assert layer.check_device_errors() == 0
        b.check(out[:-3], lse[:-3])
        nothing = b.want_lse.isinf()
        assert not out[:-3].cpu()[nothing].any()
        assert bool((out[-3:] == 5).all()) and bool((lse[-3:] == 5).all())


@pytest.mark.parametrize("fill", [math.nan, 0.0, -1.0, math.inf, -math.inf])
def test_a_block_that_nothing_began(fill):
    # its scale says nothing: new tokens in its middle are held as if they were the first
    layer = moe.PagedAttention(2, 2, 32, 32, 64, 2)
    g = torch.Generator().manual_seed(1)
    codes = torch.full((3, 2, 32, 32), 0x7f, dtype=torch.uint8, device=DEV).view(a8.F8)
    kp, vp = codes.clone(), codes.clone()
    ks, vs = (torch.full((3, 2, 2), fill, device=DEV) for _ in range(2))
    x = torch.randn(5, 2, 32, generator=g).to(BF)
    slots = [32 + 19, 32 + 20, 32 + 21, 32 + 22, 64 + 1]     # of page 1's second block, page 2
    layer.append(None, x.to(DEV), x.to(DEV), torch.zeros(5, dtype=torch.int32, device=DEV),
                 torch.tensor(slots, device=DEV), kp, vp, ac.frequencies(0).to(DEV), k_scales=ks,
                 v_scales=vs)
    assert layer.check_device_errors() == 0
    for pages, scales in ((kp, ks), (vp, vs)):
        pages, scales = pages.cpu(), scales.cpu()
        for page, block, rows, part in ((1, 1, slice(19, 23), x[:4]), (2, 0, slice(1, 2), x[4:])):
            s = a8.scale_for(part.double().abs().amax((0, 2)))
            assert torch.equal(scales[page, :, block].double(), s)
            want = a8.nearest(part.double() / s[:, None])
            assert torch.equal(pages[page, :, rows].float().double(), want.transpose(0, 1))
            pages.view(torch.uint8)[page, :, rows] = 0x7f
            scales[page, :, block] = fill
        # nothing else has changed
        assert bool((pages.view(torch.uint8) == 0x7f).all())
        assert bool(((scales == fill) | scales.isnan()).all())
