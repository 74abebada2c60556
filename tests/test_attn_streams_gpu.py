"""GPU tests of calls on a given stream: what they work on belongs to another stream,
and may be dropped as soon as the call returns."""
import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn_cases as ac

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
T, HQ, HK, D, PAGE = 700, 8, 2, 64, 16


def _tensors():
    i32 = dict(dtype=torch.int32, device=DEV)
    pages = -(-T // PAGE)
    return dict(q=torch.randn(T, HQ, D, device=DEV).to(BF), k=torch.randn(T, HK, D, device=DEV).to(BF),
                v=torch.randn(T, HK, D, device=DEV).to(BF), pos=torch.arange(T, **i32),
                slots=torch.arange(T, device=DEV), freq=ac.frequencies(D).to(DEV),
                kp=torch.randn(pages, HK, PAGE, D, device=DEV).to(BF),
                vp=torch.randn(pages, HK, PAGE, D, device=DEV).to(BF),
                table=torch.arange(pages, **i32)[None], cu=torch.tensor([0, T], **i32),
                kv=torch.tensor([T], **i32), slopes=torch.rand(HQ, device=DEV),
                prefix=torch.tensor([3], **i32), out=torch.zeros(T, HQ, D, device=DEV, dtype=BF),
                lse=torch.zeros(T, HQ, device=DEV))


CALLS = {
    "rope": (["q", "pos", "freq", "out"],
             lambda a, t, s: moe.moe_attn_rope(t["q"], t["pos"], t["freq"], out=t["out"], stream=s)),
    "append": (["q", "k", "v", "pos", "slots", "freq", "kp", "vp", "out"],
               lambda a, t, s: a.append(t["q"], t["k"], t["v"], t["pos"], t["slots"], t["kp"],
                                        t["vp"], t["freq"], q_out=t["out"], stream=s)),
    "forward": (["q", "kp", "vp", "table", "cu", "kv", "slopes", "prefix", "out", "lse"],
                lambda a, t, s: a.forward(t["q"], t["kp"], t["vp"], t["table"], t["cu"], t["kv"], T,
                                          slopes=t["slopes"], prefix=t["prefix"], out=t["out"],
                                          lse=t["lse"], stream=s)),
}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("call", list(CALLS))
def test_memory_in_use_is_not_handed_out_again(call, raw):
    names, run = CALLS[call]
    layer = moe.PagedAttention(HQ, HK, D, PAGE, T, 1)
    side = torch.cuda.Stream()
    run(layer, _tensors(), side)
    torch.cuda.synchronize()
    for name in names:
        t = _tensors()
        t[name] = t[name].clone()               # memory of its own
        address, size = t[name].data_ptr(), t[name].untyped_storage().nbytes()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(60_000_000)       # the call runs some 30 ms later
        run(layer, t, side.cuda_stream if raw else side)
        del t[name]
        new = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(4)]
        assert not side.query()
        assert address not in [n.data_ptr() for n in new], name
        side.synchronize()
