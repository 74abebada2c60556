"""GPU tests of the attention operators' handles: what a new one may be used for at
once, and what making and dropping one leaves undisturbed."""
import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn_cases as ac

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def test_a_new_handle_is_ready_for_any_stream():
    # its memory is cleared behind what the default stream still has to do, which
    # another stream does not wait for: create returns when that is over
    moe.PagedAttention(8, 2, 128, 16, 64, 4).close()      # loads the kernels
    b = ac.Batch([(40, 3000), (1, 700)], 8, 2, 128, 16, BF)
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)                        # some 0.2 s
    behind = torch.cuda.Event()
    behind.record()
    layer = moe.PagedAttention(8, 2, 128, 16, b.tokens, 2)
    assert behind.query()
    s = torch.cuda.Stream()
    out, lse = b.run(layer, stream=s)
    s.synchronize()
    b.check(out, lse)
    assert layer.check_device_errors() == 0


def test_a_layer_dropped_in_a_capture_does_not_end_it():
    import gc
    b = ac.Batch([(40, 300), (1, 70)], 8, 2, 64, 16, BF)
    layer = moe.PagedAttention(8, 2, 64, 16, b.tokens, 2)
    other = moe.PagedAttention(8, 2, 64, 16, 64, 4)
    out, lse = torch.empty_like(b.q), torch.empty(b.tokens, 8, device=DEV)
    b.run(layer, out=out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        del other
        gc.collect()
        b.run(layer, out=out, lse=lse)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    b.check(out, lse)
    assert layer.check_device_errors() == 0


@pytest.mark.parametrize("n", [1, 40])
def test_strides_of_single_elements_say_nothing(n):
    # a cache of one page and one kv head, K and V cut from differently wide buffers
    b = ac.Batch([(n, 16)], 20, 1, 64, 16, BF)
    layer = moe.PagedAttention(20, 1, 64, 16, n, 1)
    page = int(b.table[0, 0])
    b.k_pages = b.k_pages[page:page + 1].as_strided((1, 1, 16, 64), (7, 3, 64, 1))
    v = torch.zeros(1, 5, 16, 64, dtype=BF, device=DEV)
    v[:, 2] = b.v_pages[page]
    b.v_pages = v[:, 2:3]
    b.table = torch.zeros_like(b.table)
    b.check(*b.run(layer))
    assert layer.check_device_errors() == 0


@pytest.mark.parametrize("group", [1, 4, 20])
def test_new_tokens_that_max_q_does_not_allow_are_reported(group):
    b = ac.Batch([(3, 40), (0, 9), (2, 20)], group, 1, 64, 16, BF)
    layer = moe.PagedAttention(group, 1, 64, 16, b.tokens, 3)
    for max_q, flags in ((3, 0), (2, 0x2), (1, 0x2), (0, 0x2)):
        b.max_q = max_q
        out, lse = torch.full_like(b.q, 7.0), torch.full((b.tokens, group), 7.0, device=DEV)
        b.run(layer, out=out, lse=lse)
        assert layer.check_device_errors() == flags
        kept = [n > max_q for n, _ in b.lens]
        assert bool((out[:3] == 7.0).all()) == kept[0] and bool((out[3:] == 7.0).all()) == kept[2]
    # none at all: nothing to report
    b.cu_q, b.max_q = torch.zeros_like(b.cu_q), 0
    b.run(layer)
    assert layer.check_device_errors() == 0
