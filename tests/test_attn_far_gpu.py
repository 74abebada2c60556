"""GPU tests of distances that fp32 cannot count one by one: caches of more than
2^24 keys under a distance bias, on few pages that a long table repeats."""
import math

import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn_cases as ac

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.mark.parametrize("kv", [2 ** 24 + 77, 2 ** 26 + 1001])
@pytest.mark.parametrize("hq,n", [(32, 1), (4, 1), (4, 9)])   # both kernels
@pytest.mark.parametrize("slope", [-1e-4, -1e-6, 3e-8])
def test_bias_over_long_distances(kv, hq, n, slope):
    # where the bias grows with the distance the first keys have the say. A distance
    # is rounded to fp32 (2^-23 of it, twice), its bias and their sum with the score
    # too: 2^-22 of the largest bias, times log2(e) and back, below 2^-21 together
    d, page, pages = 8, 256, 8
    g = torch.Generator(device=DEV).manual_seed(5)
    q = torch.randn(n, hq, d, generator=g, device=DEV).to(BF)
    kp = torch.randn(pages, 1, page, d, generator=g, device=DEV).to(BF)
    vp = torch.randn(pages, 1, page, d, generator=g, device=DEV).to(BF)
    i32 = dict(dtype=torch.int32, device=DEV)
    columns = -(-kv // page)
    table = (torch.arange(columns, **i32) % pages)[None].contiguous()
    slopes = torch.full((hq,), slope, device=DEV) * torch.linspace(0.5, 1, hq, device=DEV)
    layer = moe.PagedAttention(hq, 1, d, page, n, 1)
    out, lse = layer.forward(q, kp, vp, table, torch.tensor([0, n], **i32),
                             torch.tensor([kv], **i32), n, slopes=slopes, return_lse=True)
    assert layer.check_device_errors() == 0
    k, v = (t.reshape(-1, d).double() for t in (kp, vp))
    j = torch.arange(kv, device=DEV)
    for i in {0, n - 1}:
        for h in (0, hq - 1):
            s = float(slopes[h])
            x = (k @ q[i, h].double() * d ** -0.5).repeat(columns * page // len(k) + 1)[:kv]
            x = x - s * (kv - n + i - j).abs()
            x[kv - n + i + 1:] = -math.inf
            want_lse = torch.logsumexp(x, 0)
            w = torch.exp(x - want_lse).reshape(-1)
            pad = torch.cat([w, w.new_zeros(-kv % len(k))]).reshape(-1, len(k)).sum(0)
            e = 1e-4 + 2.0 ** -21 * abs(s) * kv
            assert abs(float(lse[i, h]) - float(want_lse)) <= e, (i, h)
            u = ac.ROUND[BF]
            want, a = pad @ v, pad @ v.abs()
            bound = u * want.abs() + (u + math.expm1(2 * e)) * a + 2.0 ** -24
            assert bool(((out[i, h].double() - want).abs() <= bound).all()), (i, h)
