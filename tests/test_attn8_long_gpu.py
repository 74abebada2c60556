"""Calls of include/moe_attn8.h long enough for what short ones do not reach: threads that
walk along many tokens, several tokens side by side, runs whose heads a CTA takes in
turn."""
import pytest
import torch

from tests.test_attn8_gpu import BF, F32, FP, _built, test_append8 as append8  # noqa: F401
from tests.test_attn8_gpu import test_norm_rope as norm_rope
from tests.test_attn8_gpu import test_norm_rope_gradient as norm_rope_gradient

pytestmark = pytest.mark.gpu

NORMS = [
    # tokens, hq, hk, dim, rot, layout, dtype, weights, each head its own
    (20011, 1, 1, 16, 16, "half", BF, BF, False), (9001, 2, 1, 32, 16, "interleaved", FP, F32, True),
    (6007, 1, 1, 128, 128, "half", FP, FP, False), (3001, 32, 8, 128, 64, "interleaved", BF, BF, False),
    (5003, 3, 2, 80, 80, "half", BF, F32, True), (4999, 1, 2, 256, 256, "interleaved", BF, BF, True),
    (7001, 2, 1, 24, 8, "interleaved", BF, BF, False),       # half chunks: any form
]


@pytest.mark.parametrize("T,hq,hk,d,rot,layout,dtype,wide,each", NORMS)
def test_norm_rope(T, hq, hk, d, rot, layout, dtype, wide, each):
    norm_rope(T, hq, hk, d, rot, layout, dtype, wide, each)


@pytest.mark.parametrize("T,hq,hk,d,rot,layout,dtype,wide,each", NORMS)
def test_norm_rope_gradient(T, hq, hk, d, rot, layout, dtype, wide, each):
    norm_rope_gradient(T, hq, hk, d, rot, layout, dtype, wide, each)


@pytest.mark.parametrize("lens,hq,hk,d,rot,page,layout,dtype,with_norm", [
    ([(2600, 2711), (30, 55)], 8, 8, 64, 64, 32, "half", BF, True),
    ([(5000, 5003)], 5, 5, 32, 32, 16, "interleaved", FP, True),       # 10 rows of heads, by fours
    ([(1, 3), (1700, 1700), (900, 1000)], 10, 10, 16, 16, 64, "half", FP, False),
    ([(2500, 2500)], 9, 9, 40 * 2, 40, 128, "interleaved", BF, True),  # any form
])
@pytest.mark.parametrize("with_q", [True, False])
def test_append8(lens, hq, hk, d, rot, page, layout, dtype, with_norm, with_q):
    append8(lens, hq, hk, d, rot, page, layout, dtype, with_norm, with_q)
