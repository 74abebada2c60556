"""Scales of V that lie far apart: what they do to the softmax's sum, on each path over
codes."""
import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn8_cases as a8
from tests import attn_cases as ac

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.lib()


@pytest.mark.parametrize("lens", [[(1, 900), (1, 70)], [(4, 900), (3, 333)], [(40, 900), (64, 700)],
                                  [(200, 900), (150, 500)]])
@pytest.mark.parametrize("gains", [((0, 1), (-50, 51)), ((0, 1), (-55, -50)), ((0, 1), (45, 56))])
def test_scales_of_v_far_apart(lens, gains):
    # Up to 2^100 between blocks of a row: a weight below 2^(100 - 126) of another's may
    # be lost to the sum, which for 900 keys is 1.3e-5 of it, of 1e-4 here.
    b = a8.Batch8(lens, 8, 2, 128, 16, torch.bfloat16, gains=gains)
    layer = moe.PagedAttention(8, 2, 128, 16, b.tokens, len(lens))
    for kw in ({}, dict(stream=torch.cuda.current_stream())):
        out, lse = b.run(layer, **kw)
        assert layer.check_device_errors() == 0
        # numerators of bf16 on the way over 16 bits, else of fp16
        u = 2.0 ** -8
        numerator = u if lens[0][0] == 200 and not kw else 2.0 ** -11
        err = (out.cpu().double() - b.want).abs()
        assert bool(out.isfinite().all())
        assert bool((err <= u * b.want.abs() + (numerator + 1e-4) * b.bound).all())
        assert bool(((lse.cpu().double() - b.want_lse).abs() <= 1e-4 +
                     2.0 ** -22 * b.want_lse.abs()).all())
