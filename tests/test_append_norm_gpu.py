"""Norms and rotary positions on the way to a 16-bit cache (moe_attn_append_norm) against
the definition in fp64 (attn8_cases.py)."""
import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn8_cases as a8
from tests import attn_cases as ac

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
RANGE = 0x2


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.lib()


def close(got, want, slack, dtype):
    err = (got.detach().cpu().double() - want).abs()
    bound = ac.ROUND[dtype] * want.abs() + slack + 2.0 ** -24
    assert bool((err <= bound).all()), (float((err - bound).max()), int((err > bound).sum()))


class Case:
    """Tokens that go to a few rows of a cache whose other rows hold something."""

    def __init__(self, T, hq, hk, d, rot, page, layout, dtype, inner=True, wide=None, each=False,
                 offset=0, pad=0):
        g = torch.Generator().manual_seed(T + d)
        self.T, self.hq, self.hk, self.d, self.page, self.layout = T, hq, hk, d, page, layout
        self.dtype, self.rot = dtype, rot
        self.pages = -(-T // page) + 3
        shape = (self.pages, hk, page, d) if inner else (self.pages, page, hk, d)
        self.before = [torch.randn(shape, generator=g).to(dtype) for _ in "kv"]
        self.kp, self.vp = (p.clone().to(DEV) for p in self.before)
        if not inner:
            self.before = [p.transpose(1, 2) for p in self.before]
            self.kp, self.vp = self.kp.transpose(1, 2), self.vp.transpose(1, 2)
        heads = hq + 2 * hk
        buf = torch.randn(T, heads * (d + pad) + offset, generator=g).to(dtype).to(DEV)
        self.qkv = torch.as_strided(buf, (T, heads, d), (buf.stride(0), d + pad, 1), offset)
        self.host = self.qkv.cpu().clone()
        self.w = [torch.randn((h, d) if each else (d,), generator=g).to(wide or dtype)
                  for h in (hq, hk)]
        self.norm = moe.HeadNorm(self.w[0].to(DEV), self.w[1].to(DEV), 1e-5, 0.5)
        self.freq = ac.frequencies(rot)
        self.pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (T,), generator=g).to(torch.int32)
        self.slots = torch.randperm(self.pages * page, generator=g)[:T]
        self.layer = moe.PagedAttention(hq, hk, d, page, T, 4, dtype=dtype)

    def run(self, slots=None, **kw):
        q, k, v = self.qkv.split([self.hq, self.hk, self.hk], dim=1)
        args = dict(q=q, norm=self.norm, layout=self.layout, magnitude=1.25)
        args.update(kw)
        return self.layer.append(args.pop("q"), k, v, self.pos.to(DEV),
                                 (self.slots if slots is None else slots).to(DEV), self.kp,
                                 self.vp, self.freq.to(DEV), **args)

    def check(self, got, slots=None):
        slots = self.slots if slots is None else slots
        q, k, v = self.host.split([self.hq, self.hk, self.hk], dim=1)

        def turned(x, w):
            return a8.norm_rope(x, w, 0.5, 1e-5, self.pos, self.freq, self.layout, 1.25)

        if got is not None:
            close(got, *turned(q, self.w[0]), self.dtype)
        there = (slots >= 0) & (slots < self.pages * self.page)
        p, o = slots[there] // self.page, slots[there] % self.page
        want, slack = turned(k, self.w[1])
        close(self.kp.cpu()[p, :, o], want[there], slack[there], self.dtype)
        assert torch.equal(self.vp.cpu()[p, :, o], v[there])
        # and nothing else
        for now, old in zip((self.kp, self.vp), self.before):
            now, old = now.cpu().clone(), old.clone()
            now[p, :, o] = old[p, :, o] = 0
            assert torch.equal(now.view(torch.int16), old.view(torch.int16))


CASES = [
    dict(T=1, hq=32, hk=8, d=128, rot=128, page=16, layout="half", dtype=BF),
    dict(T=64, hq=32, hk=8, d=128, rot=64, page=16, layout="interleaved", dtype=BF, inner=False),
    dict(T=77, hq=6, hk=2, d=80, rot=80, page=32, layout="half", dtype=FP, wide=F32, each=True),
    dict(T=130, hq=7, hk=7, d=96, rot=24, page=64, layout="interleaved", dtype=BF, inner=False),
    dict(T=33, hq=4, hk=4, d=64, rot=0, page=128, layout="half", dtype=BF, each=True),
    dict(T=40, hq=8, hk=1, d=8, rot=8, page=256, layout="interleaved", dtype=FP),
    dict(T=19, hq=4, hk=2, d=64, rot=64, page=16, layout="half", dtype=BF, offset=1, pad=3),
    dict(T=19, hq=4, hk=2, d=64, rot=64, page=16, layout="half", dtype=FP, offset=8, pad=8),
    dict(T=5003, hq=4, hk=1, d=128, rot=128, page=16, layout="half", dtype=BF),
    dict(T=9801, hq=2, hk=2, d=64, rot=32, page=64, layout="interleaved", dtype=FP, each=True),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("with_q", [True, False])
def test_append_norm(case, with_q):
    c = Case(**case)
    got = c.run() if with_q else c.run(q=None)
    assert c.layer.check_device_errors() == 0
    assert (got is None) != with_q
    c.check(got)


def test_queries_in_place_and_on_a_given_stream():
    c = Case(50, 6, 2, 64, 64, 32, "half", BF)
    q = c.qkv[:, :6]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(q_out=q, stream=s)
    s.synchronize()
    assert got is q
    c.check(got)


def test_negative_slots_and_slots_past_the_cache():
    for case in (CASES[1], CASES[3]):        # the fast form, and any
        c = Case(**case)
        slots = c.slots.clone()
        slots[3], slots[9], slots[20] = -1, -(2 ** 40), -7
        c.check(c.run(slots=slots), slots)
        assert c.layer.check_device_errors() == 0
        slots[5], slots[11] = c.pages * c.page, 2 ** 40
        c = Case(**case)                     # (the pages as they were)
        got = c.run(slots=slots)
        assert c.layer.check_device_errors() == RANGE
        c.check(got, slots)


def test_append_norm_refusals():
    c = Case(5, 4, 2, 64, 64, 16, "half", BF)
    w = c.norm.q_weight
    for bad in (moe.HeadNorm(w[:32], w), moe.HeadNorm(w, w.half()), moe.HeadNorm(w.cpu(), w),
                moe.HeadNorm(w, w.expand(2, 64)), moe.HeadNorm(w, None), (w, w, 1e-6, 0.0)):
        with pytest.raises((ValueError, AttributeError)):
            c.run(norm=bad)
    with pytest.raises(ValueError, match="no_grad"):
        c.run(norm=moe.HeadNorm(w, w.clone().requires_grad_()))
    for eps in (-1.0, float("inf"), float("nan")):
        with pytest.raises(moe.MoeError):
            c.run(norm=moe.HeadNorm(w, w, eps))
    with pytest.raises(moe.MoeError):        # queries onto keys
        c.run(q_out=c.qkv[:, 1:5])
    for now, old in zip((c.kp, c.vp), c.before):
        assert torch.equal(now.cpu(), old)
