"""What the attention kernels do once a wait has given up. No wait is made to hang
here: the handle's error word is set by hand, after which every wait that is not
over at once gives up by itself, as after a real timeout."""
import ctypes

import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn_cases as ac
from w4a16_routed_expert_router_gb300 import attention as at

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16


class _Words:
    def __init__(self, address, n):
        self.__cuda_array_interface__ = {"data": (address, False), "shape": (n,),
                                         "typestr": "<i4", "version": 2}


def _error_word(layer):
    """The first word of the handle's workspace, as a tensor."""
    ws = ctypes.c_void_p.from_address(layer.handle.value + ctypes.sizeof(at.moe_attn_config) + 8)
    word = torch.as_tensor(_Words(ws.value, 1), device=DEV)
    word.fill_(at.MOE_ATTN_DEVERR_RANGE)
    assert layer.check_device_errors() == at.MOE_ATTN_DEVERR_RANGE  # it is that word
    assert layer.check_device_errors() == 0
    return word


CASES = [  # hq, hk, d, page, dtype, [(new tokens, keys)], scores
    (32, 8, 128, 16, BF, [(40, 30001)], {}),                       # cut in step, joined
    (8, 2, 128, 64, BF, [(700, 5001), (1, 9000), (90, 77)], {}),
    (16, 4, 64, 32, FP, [(300, 7003), (64, 9001)], {}),
    (12, 4, 96, 16, BF, [(500, 2011), (260, 4001), (1, 333)], dict(softcap=20.0, window=900)),
    (8, 8, 128, 16, BF, [(1, 20000), (1, 333), (1, 15000)], {}),   # the few-token kernel
]


@pytest.mark.parametrize("hq,hk,d,page,dtype,lens,kw", CASES)
def test_launches_end_and_the_timeout_is_reported(hq, hk, d, page, dtype, lens, kw):
    b = ac.Batch(lens, hq, hk, d, page, dtype, **kw)
    layer = moe.PagedAttention(hq, hk, d, page, b.tokens, len(lens), dtype=dtype)
    out, lse = b.run(layer)
    b.check(out, lse)
    word = _error_word(layer)
    word.fill_(at.MOE_ATTN_DEVERR_TIMEOUT)
    for _ in range(5):
        b.run(layer)
    assert layer.check_device_errors() == at.MOE_ATTN_DEVERR_TIMEOUT
    assert layer.check_device_errors() == 0


@pytest.mark.parametrize("hq,hk,d,page,dtype,lens,kw", CASES)
def test_results_after_a_timeout_are_right_again(hq, hk, d, page, dtype, lens, kw):
    b = ac.Batch(lens, hq, hk, d, page, dtype, **kw)
    layer = moe.PagedAttention(hq, hk, d, page, b.tokens, len(lens), dtype=dtype)
    out, lse = b.run(layer)
    word = _error_word(layer)
    for _ in range(3):
        word.fill_(at.MOE_ATTN_DEVERR_TIMEOUT)
        b.run(layer)
        assert layer.check_device_errors() == at.MOE_ATTN_DEVERR_TIMEOUT
        for _ in range(3):
            o2, l2 = b.run(layer)
            assert torch.equal(o2, out) and torch.equal(l2, lse)
        assert layer.check_device_errors() == 0
