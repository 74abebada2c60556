"""Appending long prompts of layers with few query heads to the 8-bit cache: queries walk
along the tokens several side by side, with a table for each, which is when a launch asks
for most shared memory."""
import pytest

from tests.test_attn8_gpu import BF, FP, _built, test_append8 as append8  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,hq,hk,d,rot,page,layout,dtype,with_norm", [
    (8192, 4, 1, 128, 128, 16, "half", BF, True),
    (4864, 1, 1, 128, 128, 32, "interleaved", FP, True),
    (4863, 4, 2, 128, 128, 64, "half", FP, False),            # one token less than that takes
    (9800, 4, 1, 64, 64, 64, "half", FP, True),
    (9800, 2, 1, 128, 64, 16, "interleaved", BF, False),
    (19500, 4, 1, 32, 32, 16, "half", BF, True),
    (19500, 1, 1, 128, 32, 256, "half", FP, True),
    (39000, 2, 1, 32, 16, 128, "interleaved", BF, True),
    (39000, 4, 4, 16, 16, 16, "half", FP, False),
])
def test_long_prompts_of_few_heads(T, hq, hk, d, rot, page, layout, dtype, with_norm):
    append8([(T, T)], hq, hk, d, rot, page, layout, dtype, with_norm, True)
