"""Attention over the 8-bit cache of batches that mix single tokens, parts of a tile and
chunks, against the definition in fp64 (attn8_cases.py)."""
import ctypes

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


@pytest.mark.parametrize("d,dtype,opt", [(128, BF, {}), (64, FP, {}), (128, FP, dict(softcap=30.0)),
                                         (96, BF, dict(window=300, sinks=5))])
def test_single_tiles_in_front_of_pairs_of_tiles(d, dtype, opt):
    # items of one tile (up to 32 tokens at a group of 4), which the other tile's warps
    # pass over, in front of items of two, over blocks whose scales differ: a row that is
    # given another block's scales is off by factors
    lens = []
    for i in range(40):
        lens += [((1, 3, 32)[i % 3], 900 - 13 * i), ((33, 64, 50)[i % 3], 64 + 17 * i)]
    b = a8.Batch8(lens, 16, 4, d, 16, dtype, gains=((-3, 3), (-6, 7)), scale=0.05, **opt)
    layer = moe.PagedAttention(16, 4, d, 16, b.tokens, len(lens), dtype=dtype)
    out, lse = b.run(layer)
    assert layer.check_device_errors() == 0
    # numerators in fp16, scores up to 2^3 of the plain ones' size
    u = ac.ROUND[dtype]
    err = (out.cpu().double() - b.want).abs()
    bound = u * b.want.abs() + (2.0 ** -11 + 8e-4) * b.bound + 2.0 ** -24
    assert bool((err <= bound).all()), float((err / bound).max())
    assert bool(((lse.cpu().double() - b.want_lse).abs() <= 8e-4).all())
    for _ in range(30):
        again, lse2 = b.run(layer)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
    assert layer.check_device_errors() == 0


def scratch_bytes(layer, b):
    n = ctypes.c_size_t()
    batch = moe.attention.moe_attn_batch(None, None, None, b.table.shape[1], b.table.shape[1],
                                         len(b.lens), b.tokens, b.max_q)
    assert layer._library.moe_attn_forward8_scratch_bytes(layer.handle, batch, n) == 0
    return n.value


@pytest.mark.parametrize("lens,brought", [
    ([(1, 1000), (380, 900), (1, 77), (2, 130)], False), ([(1, 1000), (382, 900), (1, 77)], False),
    ([(1, 1000), (383, 900), (1, 77)], True), ([(1, 1000), (700, 900), (1, 77)], True)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_chunks_beside_single_tokens_on_both_sides_of_the_rule(lens, brought, dtype):
    # more than 512 rows to a sequence and kv head, on average, bring the keys to 16 bits
    b = a8.Batch8(lens, 8, 2, 128, 32, dtype)
    layer = moe.PagedAttention(8, 2, 128, 32, b.tokens, len(lens), dtype=dtype)
    assert (b.tokens * 4 > 512 * len(lens)) == (scratch_bytes(layer, b) > 0) == brought
    for kw in ({}, dict(stream=torch.cuda.current_stream())):   # on a given one: over codes
        out, lse = b.run(layer, **kw)
        assert layer.check_device_errors() == 0
        b.check(out, lse)
