"""Keys and values of an fp16 layer next to the largest that fp16 has: codes bring them
above it, and they stay finite wherever they come back to 16 bits."""
import math

import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn8_cases as a8
from tests import attn_cases as ac

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FP, TOP = torch.float16, 65504.0


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.lib()


def appended(n, d, page, g):
    """A layer of one head, its cache on the device after n tokens, and the cache in fp64:
    from token 64 on, some keys and values are 60000 to 65504."""
    layer = moe.PagedAttention(1, 1, d, page, n, 1, dtype=FP)
    x = [torch.randn(n, 1, d, generator=g) for _ in range(2)]
    for t in x:
        big = torch.rand(n, 1, d, generator=g) < 0.2
        big[:64] = False
        top = 60000 + 5504 * torch.rand(n, 1, d, generator=g)
        t.copy_(torch.where(big, torch.copysign(top, t), t * 30))
        t[70, 0, :4] = torch.tensor([TOP, -TOP, 63488.0, 63456.0])
    k, v = (t.to(FP) for t in x)
    pages = -(-n // page)
    cache = a8.Cache(pages, 1, page, d, g)
    dev = cache.on(DEV)
    layer.append(None, k.to(DEV), v.to(DEV), torch.zeros(n, dtype=torch.int32, device=DEV),
                 torch.arange(n, device=DEV), dev[0], dev[1], ac.frequencies(0).to(DEV),
                 k_scales=dev[2], v_scales=dev[3])
    cache.append("k", k.double(), list(range(n)))
    cache.append("v", v.double(), list(range(n)))
    held = [cache.held(h).transpose(1, 2).reshape(-1, 1, d)[:n] for h in "kv"]
    assert all(float(h.abs().max()) == 65536.0 for h in held)
    return layer, dev, held


@pytest.mark.parametrize("d,page", [(128, 16), (64, 64)])
def test_values_next_to_the_top_come_back_finite(d, page):
    n = 200
    layer, dev, held = appended(n, d, page, torch.Generator().manual_seed(d))
    dev[0].view(torch.uint8)[0, 0, 3, 5] = 0x7f        # what is no number stays none
    table = torch.arange(-(-n // page), dtype=torch.int32, device=DEV)[None]
    got = layer.read(dev[0], dev[1], table, torch.tensor([0, n], dtype=torch.int32, device=DEV),
                     torch.zeros(1, dtype=torch.int32, device=DEV), n, k_scales=dev[2],
                     v_scales=dev[3])
    assert bool(got[0][3, 0, 5].isnan()) and int(got[0].isnan().sum()) == 1
    held[0][3, 0, 5] = 0.0
    got[0][3, 0, 5] = 0.0
    for x, want in zip(got, held):
        assert torch.equal(x.cpu().double(), want.clamp(-TOP, TOP).to(FP).double())
    assert float(got[0][70, 0, 0]) == TOP and float(got[0][70, 0, 1]) == -TOP


@pytest.mark.parametrize("d,page", [(128, 16), (64, 64)])
def test_attention_to_values_next_to_the_top(d, page):
    n, g = 600, torch.Generator().manual_seed(d + 1)
    layer, dev, (k, v) = appended(n, d, page, g)
    # products of about 4, as keys of 65504 have with such queries
    q = (torch.randn(n, 1, d, generator=g) * 2.0 ** -14).to(FP)
    table = torch.arange(-(-n // page), dtype=torch.int32, device=DEV)[None]
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    for kw, top in (({}, TOP), (dict(stream=torch.cuda.current_stream()), math.inf)):
        out, lse = layer.forward(q.to(DEV), dev[0], dev[1], table, cu, cu[1:], n, return_lse=True,
                                 k_scales=dev[2], v_scales=dev[3], **kw)
        assert layer.check_device_errors() == 0
        want, bound, want_lse = a8.sequence(q, k.clamp(-top, top), v.clamp(-top, top), d ** -0.5)
        # one rounding of the result, one of each numerator, and scores of four times the
        # plain ones' size in fp32
        err = (out.cpu().double() - want).abs()
        assert bool(out.isfinite().all())
        assert bool((err <= 2.0 ** -11 * want.abs() + (2.0 ** -11 + 4e-4) * bound).all())
        assert bool(((lse.cpu().double() - want_lse).abs() <= 4e-4).all())
