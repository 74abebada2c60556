"""GPU tests of how the attention operators stand to autograd: none of them has a
formula there, so tensors that ask for a gradient are refused instead of losing it,
and tensors that are written to count as changed."""
import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn_cases as ac

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
T, HQ, HK, D, PAGE = 5, 8, 2, 64, 16


class Calls:
    def __init__(self):
        g = torch.Generator(device=DEV).manual_seed(1)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device=DEV).to(BF)

        i32 = dict(dtype=torch.int32, device=DEV)
        self.layer = moe.PagedAttention(HQ, HK, D, PAGE, T, 2)
        self.freq, self.pos = ac.frequencies(D).to(DEV), torch.arange(T, **i32)
        self.t = dict(q=normal(T, HQ, D), k=normal(T, HK, D), v=normal(T, HK, D),
                      k_pages=normal(2, HK, PAGE, D), v_pages=normal(2, HK, PAGE, D),
                      out=normal(T, HQ, D), lse=torch.zeros(T, HQ, device=DEV),
                      slopes=torch.zeros(HQ, device=DEV))
        self.slots = torch.arange(T, device=DEV)
        self.batch = (torch.zeros(1, 1, **i32), torch.tensor([0, T], **i32),
                      torch.tensor([T], **i32), T)

    def rope(self):
        return moe.moe_attn_rope(self.t["q"], self.pos, self.freq, out=self.t["out"])

    def append(self):
        t = self.t
        return self.layer.append(t["q"], t["k"], t["v"], self.pos, self.slots, t["k_pages"],
                                 t["v_pages"], self.freq, q_out=t["out"])

    def forward(self):
        t = self.t
        return self.layer.forward(t["q"], t["k_pages"], t["v_pages"], *self.batch, out=t["out"],
                                  lse=t["lse"], slopes=t["slopes"])


READS = {"rope": ["q", "out"], "append": ["q", "k", "v", "k_pages", "v_pages", "out"],
         "forward": ["q", "k_pages", "v_pages", "out", "lse", "slopes"]}
WRITES = {"rope": ["out"], "append": ["out"], "forward": ["out", "lse"]}  # of given outputs


@pytest.mark.parametrize("call,name", [(c, n) for c in READS for n in READS[c]])
def test_tensors_that_ask_for_a_gradient_are_refused(call, name):
    c = Calls()
    plain = getattr(c, call)().clone()
    was = {n: t.clone() for n, t in c.t.items()}
    c.t[name].requires_grad_(True)
    with pytest.raises(ValueError, match="no_grad"):
        getattr(c, call)()
    for n, t in c.t.items():
        assert torch.equal(t.detach(), was[n])
    with torch.no_grad():
        again = getattr(c, call)()
    assert torch.equal(again, plain) and not (again.requires_grad and name != "out")


@pytest.mark.parametrize("call", list(WRITES))
def test_what_is_written_counts_as_changed(call):
    c = Calls()
    before = {n: t._version for n, t in c.t.items()}
    for mode in (torch.enable_grad, torch.no_grad):
        with mode():
            getattr(c, call)()
        for n, t in c.t.items():
            assert (t._version > before[n]) == (n in WRITES[call]), n
        before = {n: t._version for n, t in c.t.items()}


def test_a_backward_pass_that_kept_an_overwritten_tensor_raises():
    x = torch.randn(T, HQ, D, device=DEV).to(BF)
    w = torch.ones(D, device=DEV, dtype=BF, requires_grad=True)
    y = (x * w).sum()                      # keeps x for the gradient of w
    moe.moe_attn_rope(x, torch.arange(T, dtype=torch.int32, device=DEV),
                      ac.frequencies(D).to(DEV), out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@pytest.mark.parametrize("call", list(WRITES))
def test_inference_tensors_pass(call):
    with torch.inference_mode():
        c = Calls()
        inside = getattr(c, call)().clone()
    assert torch.equal(getattr(c, call)(), inside)   # outside too, where they keep no count
