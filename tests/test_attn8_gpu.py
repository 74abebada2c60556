"""GPU tests of include/moe_attn8.h against the definitions in fp64
(attn8_cases.py, which derives the bounds)."""
import math

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


# ------------------------------------------------------------------ norm and rotation
NORMS = [
    # tokens, hq, hk, dim, rot, layout, dtype, weights, each head its own
    (1, 32, 8, 128, 128, "half", BF, BF, False), (7, 3, 1, 128, 64, "interleaved", FP, F32, True),
    (65, 5, 5, 96, 24, "half", BF, F32, False), (33, 1, 1, 80, 40, "half", FP, FP, True),
    (5, 2, 1, 256, 256, "half", BF, BF, True), (4, 9, 3, 256, 256, "interleaved", FP, F32, False),
    (3, 2, 2, 6, 2, "half", BF, BF, False), (3, 2, 1, 5, 4, "interleaved", FP, F32, True),
    (9, 3, 3, 64, 0, "half", BF, BF, False), (301, 4, 2, 64, 64, "interleaved", BF, BF, True),
    (2, 300, 4, 8, 8, "half", FP, FP, True), (2, 1, 1, 255, 254, "half", BF, F32, False),
    (2, 1, 1, 1, 0, "half", FP, FP, False), (1303, 12, 4, 64, 32, "half", BF, F32, True),
    (700, 64, 8, 128, 96, "half", FP, FP, False), (1, 1, 1, 256, 0, "interleaved", BF, BF, False),
]


def norm_case(T, hq, hk, d, rot, dtype, wide, each, seed=0):
    g = torch.Generator().manual_seed(T + d + seed)
    q, k = (torch.randn(T, h, d, generator=g).to(dtype) for h in (hq, hk))
    w = [(torch.randn((h, d) if each else (d,), generator=g)).to(wide) for h in (hq, hk)]
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (T,), generator=g).to(torch.int32)
    return g, q, k, w, pos, ac.frequencies(rot)


@pytest.mark.parametrize("T,hq,hk,d,rot,layout,dtype,wide,each", NORMS)
def test_norm_rope(T, hq, hk, d, rot, layout, dtype, wide, each):
    _, q, k, w, pos, freq = norm_case(T, hq, hk, d, rot, dtype, wide, each)
    norm = moe.HeadNorm(w[0].to(DEV), w[1].to(DEV), 1e-5, 0.5)
    got = moe.moe_attn_norm_rope(q.to(DEV), k.to(DEV), pos.to(DEV), freq.to(DEV), norm,
                                 layout=layout, magnitude=1.25)
    for x, wx, y in zip((q, k), w, got):
        want, slack = a8.norm_rope(x, wx, 0.5, 1e-5, pos, freq, layout, 1.25)
        close(y, want, slack, dtype)
    alone = moe.moe_attn_norm_rope(None, k.to(DEV), pos.to(DEV), freq.to(DEV), norm, layout=layout,
                                   magnitude=1.25)
    assert alone[0] is None and torch.equal(alone[1], got[1])


@pytest.mark.parametrize("T,hq,hk,d,rot,layout,dtype,wide,each", NORMS)
def test_norm_rope_gradient(T, hq, hk, d, rot, layout, dtype, wide, each):
    g, q, k, w, pos, freq = norm_case(T, hq, hk, d, rot, dtype, wide, each)
    dq, dk = (torch.randn(x.shape, generator=g).to(dtype) for x in (q, k))
    norm = moe.HeadNorm(w[0].to(DEV), w[1].to(DEV), 1e-5, 0.5)
    args = [x.to(DEV) for x in (dq, dk, q, k, pos, freq)]
    got = moe.moe_attn_norm_rope_backward(*args, norm, layout=layout, magnitude=1.25)
    again = moe.moe_attn_norm_rope_backward(*args, norm, layout=layout, magnitude=1.25)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for i, (dy, x, wx) in enumerate(((dq, q, w[0]), (dk, k, w[1]))):
        dx, slack, dw, wslack = a8.norm_rope_gradient(dy, x, wx, 0.5, 1e-5, pos, freq, layout, 1.25)
        close(got[i], dx, slack, dtype)
        if not each:
            dw, wslack = dw.sum(0), wslack.sum(0)
        assert got[2 + i].dtype == F32 and got[2 + i].shape == dw.shape
        err = (got[2 + i].cpu().double() - dw).abs()
        assert bool((err <= wslack).all()), float((err / wslack).max())
    alone = moe.moe_attn_norm_rope_backward(args[0], None, args[2], None, *args[4:], norm,
                                            layout=layout, magnitude=1.25)
    assert alone[1] is None and alone[3] is None and torch.equal(alone[0], got[0])


def test_norm_gradient_against_differences():
    # L = <g, y(x, w)> in single coordinates of x and w: the formula's gradient
    # against central differences in fp64, the kernel's against the formula's (above)
    T, H, D = 4, 2, 32
    g, q, _, w, pos, freq = norm_case(T, H, 1, D, 16, FP, F32, True)
    dy = torch.randn(T, H, D, generator=g).to(FP)
    dx, slack, dw, wslack = a8.norm_rope_gradient(dy, q, w[0], 0.5, 1e-5, pos, freq, "half")
    got = moe.moe_attn_norm_rope_backward(dy.to(DEV), None, q.to(DEV), None, pos.to(DEV),
                                          freq.to(DEV), moe.HeadNorm(w[0].to(DEV), None, 1e-5, 0.5))

    def loss(x, weight):
        y = a8.normed(x, weight, 0.5, 1e-5)[0]
        return float((dy.double() * ac.rotary(y, pos, freq, "half")[0]).sum())

    step = 2.0 ** -12
    for t, h, i in ((0, 0, 0), (1, 1, 9), (3, 0, 31), (2, 1, 16)):
        e = torch.zeros(T, H, D, dtype=torch.float64)
        e[t, h, i] = step
        d = (loss(q.double() + e, w[0]) - loss(q.double() - e, w[0])) / (2 * step)
        assert abs(d - float(dx[t, h, i])) < 1e-4          # step^2 times third derivatives
        assert abs(d - float(got[0][t, h, i])) < 1e-4 + 2.0 ** -11 * abs(d) + float(slack[t, h, i])
        d = (loss(q, w[0].double() + e[0]) - loss(q, w[0].double() - e[0])) / (2 * step)
        if t == 0:
            assert abs(d - float(got[2][h, i])) < 1e-6 + float(wslack[h, i])


@pytest.mark.parametrize("offset,pad", [(0, 0), (4, 4), (1, 3), (8, 8)])
def test_norm_rope_strided_in_place(offset, pad):
    T, H, D = 19, 6, 64
    buf = torch.randn(T, H * (D + pad) + offset, device=DEV).to(BF)
    view = torch.as_strided(buf, (T, H, D), (buf.stride(0), D + pad, 1), offset)
    before, x = buf.clone(), view.clone()
    pos = torch.arange(100, 100 + T, dtype=torch.int32, device=DEV)
    freq = ac.frequencies(D)
    w = torch.rand(D, device=DEV).to(BF)
    q, k = view[:, :4], view[:, 4:]
    got = moe.moe_attn_norm_rope(q, k, pos, freq.to(DEV), moe.HeadNorm(w, w), q_out=q, k_out=k)
    assert got[0] is q and got[1] is k
    want, slack = a8.norm_rope(x, w, 0.0, 1e-6, pos, freq, "half")
    close(view, want, slack, BF)
    touched = torch.zeros(buf.numel(), dtype=torch.bool, device=DEV)
    torch.as_strided(touched, (T, H, D), (buf.stride(0), D + pad, 1), offset).fill_(True)
    assert torch.equal(buf.flatten()[~touched], before.flatten()[~touched])


def test_norm_rope_empty_zero_rows_and_streams():
    freq = ac.frequencies(64).to(DEV)
    w = torch.rand(64, device=DEV)
    norm = moe.HeadNorm(w, w)
    e, pos0 = torch.empty(0, 4, 64, dtype=BF, device=DEV), torch.empty(0, dtype=torch.int32,
                                                                       device=DEV)
    out = moe.moe_attn_norm_rope(e, e, pos0, freq, norm)
    assert out[0].shape == out[1].shape == (0, 4, 64)
    back = moe.moe_attn_norm_rope_backward(e, e, e, e, pos0, freq, norm)
    assert not back[2].any() and not back[3].any() and back[2].shape == (64,)
    # a row of zeros: eps alone under the root
    x = torch.zeros(5, 2, 64, dtype=BF, device=DEV)
    pos = torch.arange(5, dtype=torch.int32, device=DEV)
    assert not moe.moe_attn_norm_rope(x, None, pos, freq, norm)[0].any()
    dy = torch.ones_like(x)
    back = moe.moe_attn_norm_rope_backward(dy, None, x, None, pos, freq, norm)
    want = a8.norm_rope_gradient(dy, x, w.cpu(), 0.0, 1e-6, pos.cpu(), freq.cpu(), "half")
    close(back[0], want[0], want[1], BF)
    # another stream
    x = torch.randn(50, 4, 64, device=DEV).to(BF)
    pos = torch.arange(50, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.moe_attn_norm_rope(x, x, pos, freq, norm, stream=s)
    back = moe.moe_attn_norm_rope_backward(x, None, x, None, pos, freq, norm, stream=s)
    s.synchronize()
    assert torch.equal(got[0], moe.moe_attn_norm_rope(x, None, pos, freq, norm)[0])
    assert torch.equal(back[2], moe.moe_attn_norm_rope_backward(x, None, x, None, pos, freq,
                                                                norm)[2])
    with pytest.raises(ValueError):
        moe.moe_attn_norm_rope(x, x, pos, freq, norm, stream=s.cuda_stream)


def test_norm_rope_refuses_gradients_and_wrong_weights():
    x = torch.randn(3, 2, 64, device=DEV).to(BF)
    pos, freq = torch.arange(3, dtype=torch.int32, device=DEV), ac.frequencies(64).to(DEV)
    w = torch.ones(64, device=DEV)
    for bad in (x.clone().requires_grad_(), ):
        with pytest.raises(ValueError, match="moe_attn_norm_rope_backward"):
            moe.moe_attn_norm_rope(bad, None, pos, freq, moe.HeadNorm(w, w))
    with pytest.raises(ValueError, match="no_grad"):
        moe.moe_attn_norm_rope(x, None, pos, freq, moe.HeadNorm(w.requires_grad_(), None))
    w = w.detach()
    for bad in (w[:32], w.half(), w.cpu(), w.repeat(3, 1), w.repeat(2, 2)[:, ::2], w[None, None]):
        with pytest.raises(ValueError):
            moe.moe_attn_norm_rope(x, None, pos, freq, moe.HeadNorm(bad, None))
    with pytest.raises(ValueError, match="one type"):
        moe.moe_attn_norm_rope(x, x, pos, freq, moe.HeadNorm(w, w.to(BF)))
    with pytest.raises(ValueError):
        moe.moe_attn_norm_rope(x, x[:2], pos, freq, moe.HeadNorm(w, w))
    with pytest.raises(ValueError):
        moe.moe_attn_norm_rope_backward(x, None, None, x, pos, freq, moe.HeadNorm(w, w))
    with pytest.raises(moe.MoeError):
        moe.moe_attn_norm_rope(x, None, pos, freq, moe.HeadNorm(w, w), q_out=x.flip(0)[:1].expand(
            3, 2, 64))


# ------------------------------------------------------------------ the 8-bit cache
def slots_of(lens, page, columns, order):
    """Slots and positions of new tokens: (new, keys) of each sequence, whose pages are
    rows of `order`."""
    slots, pos = [], []
    for s, (n, kv) in enumerate(lens):
        for p in range(kv - n, kv):
            slots.append(int(order[s, p // page]) * page + p % page)
            pos.append(p)
    return slots, pos


APPENDS = [
    # (new, keys) of each sequence, hq, hk, dim, rot, page, layout, dtype, norm
    ([(1, 1)], 4, 1, 128, 128, 16, "half", BF, True),
    ([(1, 17), (1, 16), (1, 33), (1, 48), (1, 5)], 32, 8, 128, 128, 16, "half", BF, True),
    ([(40, 77), (1, 9), (3, 3), (70, 100)], 6, 2, 80, 80, 32, "half", FP, False),
    ([(130, 130), (7, 61)], 7, 7, 96, 24, 64, "interleaved", BF, True),
    ([(17, 300)], 64, 1, 16, 16, 256, "interleaved", FP, True),
    ([(33, 40), (5, 128)], 4, 4, 64, 0, 128, "half", BF, True),
    ([(259, 700)], 3, 3, 112, 20, 16, "half", FP, True),     # chunks of 10: any form
    ([(64, 128)], 8, 8, 128, 64, 64, "half", BF, False),     # part of a head turned
    ([(1, 1 + 7 * i) for i in range(75)], 8, 2, 64, 64, 32, "interleaved", FP, True),
]


@pytest.mark.parametrize("lens,hq,hk,d,rot,page,layout,dtype,with_norm", APPENDS)
@pytest.mark.parametrize("with_q", [True, False])
def test_append8(lens, hq, hk, d, rot, page, layout, dtype, with_norm, with_q):
    g = torch.Generator().manual_seed(d + page)
    T = sum(n for n, _ in lens)
    columns = max(-(-kv // page) for _, kv in lens)
    pages = len(lens) * columns + 2
    order = torch.randperm(pages, generator=g)[:len(lens) * columns].view(len(lens), columns)
    slots, at = slots_of(lens, page, columns, order)
    cache = a8.Cache(pages, hk, page, d, g)
    qkv = torch.randn(T, hq + 2 * hk, d, generator=g).to(dtype)
    # values of very different sizes: some blocks grow, some do not
    qkv[:, hq + hk:] *= torch.pow(2.0, torch.randint(-6, 7, (T, 1, 1), generator=g)).to(dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    w = [torch.rand(d, generator=g).to(dtype) + 0.5 for _ in range(2)]
    freq, pos = ac.frequencies(rot), torch.tensor(at, dtype=torch.int32)
    layer = moe.PagedAttention(hq, hk, d, page, max(T, 1), len(lens), dtype=dtype)
    dev = cache.on(DEV)
    norm = moe.HeadNorm(w[0].to(DEV), w[1].to(DEV), 1e-5, 0.25) if with_norm else None
    gpu = qkv.to(DEV)
    got = layer.append(gpu[:, :hq] if with_q else None, gpu[:, hq:hq + hk], gpu[:, hq + hk:],
                       pos.to(DEV), torch.tensor(slots, device=DEV), dev[0], dev[1], freq.to(DEV),
                       layout=layout, norm=norm, k_scales=dev[2], v_scales=dev[3])
    assert layer.check_device_errors() == 0

    def turned(x, weight):
        if with_norm:
            return a8.norm_rope(x, weight, 0.25, 1e-5, pos, freq, layout)
        return ac.rotary(x, pos, freq, layout)

    if with_q:
        close(got, *turned(q, w[0]), dtype)
    else:
        assert got is None
    kx, kslack = turned(k, w[1])
    cache.append("k", kx, slots)
    cache.append("v", v.double(), slots)
    # scales, and V and what the blocks of K held: equal
    assert torch.equal(dev[2].cpu(), cache.scales["k"])
    assert torch.equal(dev[3].cpu(), cache.scales["v"])
    assert torch.equal(dev[1].cpu().view(torch.uint8), cache.values["v"].view(torch.uint8))
    new = torch.zeros(pages * page, dtype=torch.bool)
    new[slots] = True
    new = new.view(pages, 1, page, 1).expand_as(cache.values["k"])
    same = dev[0].cpu().view(torch.uint8) == cache.values["k"].view(torch.uint8)
    assert bool(same[~new].all())
    # new keys: half a step of the codes at the value, and its own fp32 error
    p, o = torch.tensor(slots) // page, torch.tensor(slots) % page
    s = cache.scales["k"].double()[p, :, o // 16][..., None]
    held = dev[0].cpu().view(torch.uint8)[p, :, o].view(a8.F8).float().double() * s
    bound = a8.half_step((kx.abs() + kslack) / s) * s + kslack
    assert bool(((held - kx).abs() <= bound).all())
    assert bool((same | ~new).float().mean() > 0.999)      # and off by one only at a border
    layer.close()


def test_append8_ignores_what_a_block_held_before_it_begins():
    # a recycled page: scales and codes of NaN, and scales that were never set
    layer = moe.PagedAttention(2, 2, 32, 16, 64, 2)
    g = torch.Generator().manual_seed(1)
    freq = ac.frequencies(32).to(DEV)
    for fill in (math.nan, 0.0, -1.0, math.inf):
        codes = torch.full((4, 2, 16, 32), 0x7f, dtype=torch.uint8, device=DEV).view(a8.F8)
        kp, vp = codes.clone(), codes.clone()
        ks, vs = (torch.full((4, 2, 1), fill, device=DEV) for _ in range(2))
        k = torch.randn(20, 2, 32, generator=g).to(BF)
        pos = torch.arange(20, dtype=torch.int32, device=DEV)
        # 16 tokens begin page 2, 4 go to rows 3.. of page 1, which nothing began
        slots = torch.tensor(list(range(32, 48)) + list(range(19, 23)), device=DEV)
        layer.append(None, k.to(DEV), k.to(DEV), pos, slots, kp, vp, freq, k_scales=ks, v_scales=vs)
        want = a8.quantised(k[:16])
        assert torch.equal(vs[2].cpu()[:, 0].double(), want[1][0])
        got = vp[2].float().cpu().double() * vs[2].cpu().double()[..., None]
        assert torch.equal(got.transpose(0, 1), want[2])
        top = k[16:].double().abs().amax((0, 2))
        assert torch.equal(vs[1].cpu()[:, 0].double(), a8.scale_for(top)) or fill == math.inf
        assert bool((vp[0].view(torch.uint8) == 0x7f).all())
    assert layer.check_device_errors() == 0


def test_append8_slots_out_of_range_padding_and_values_that_are_no_numbers():
    layer = moe.PagedAttention(2, 1, 64, 16, 64, 2)
    g = torch.Generator().manual_seed(2)
    freq = ac.frequencies(0).to(DEV)
    cache = a8.Cache(3, 1, 16, 64, g)
    dev = cache.on(DEV)
    v = torch.randn(12, 1, 64, generator=g).to(BF)
    v[0, 0, 3], v[1, 0, 5], v[2, 0, 7], v[7] = math.nan, math.inf, -math.inf, 0.0
    v[8] *= 2.0 ** 100
    v[9] *= 2.0 ** -100
    slots = [5, 6, 7, 8, -1, 48, -5, 16, 40, 41, 2 ** 40, -1]
    pos = torch.zeros(12, dtype=torch.int32, device=DEV)
    layer.append(None, v.to(DEV), v.to(DEV), pos, torch.tensor(slots, device=DEV), dev[0], dev[1],
                 freq, k_scales=dev[2], v_scales=dev[3])
    assert layer.check_device_errors() == RANGE
    inside = [s if 0 <= s < 48 else -1 for s in slots]
    for half in "kv":
        cache.append(half, v.double(), inside)
    for i, half in enumerate("kv"):
        assert torch.equal(dev[2 + i].cpu(), cache.scales[half])
        a, b = dev[i].cpu().float(), cache.values[half].float()
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


def test_append8_scales_that_are_no_powers_of_two():
    # a cache that another program filled: codes go by the ratio, values by division
    layer = moe.PagedAttention(2, 2, 64, 32, 64, 2)
    g = torch.Generator().manual_seed(3)
    cache = a8.Cache(2, 2, 32, 64, g)
    for half in "kv":
        cache.scales[half] = torch.rand(cache.scales[half].shape, generator=g) * 0.01 + 0.001
    dev = cache.on(DEV)
    for first, gain in ((3, 0.01), (9, 40.0)):   # within the scale, and above it
        v = (torch.randn(4, 2, 64, generator=g) * gain).to(BF)
        slots = [first, first + 1, first + 2, 32 + first]
        layer.append(None, v.to(DEV), v.to(DEV), torch.zeros(4, dtype=torch.int32, device=DEV),
                     torch.tensor(slots, device=DEV), dev[0], dev[1], ac.frequencies(0).to(DEV),
                     k_scales=dev[2], v_scales=dev[3])
        cache.append("v", v.double(), slots)
        assert torch.equal(dev[3].cpu(), cache.scales["v"])
        got, want = dev[1].cpu().float().double(), cache.values["v"].float().double()
        # x / s in fp32 may fall on the other side of a border
        assert float((got != want).double().mean()) < 1e-3
        assert bool(((got - want).abs() <= 2 * a8.half_step(want) + 1e-30).all())
        cache.values["v"] = dev[1].cpu()
    assert layer.check_device_errors() == 0


@pytest.mark.parametrize("lens,hk,d,page,dtype,inner", [
    ([(0, 5)], 1, 128, 16, BF, True), ([(3, 40), (7, 0), (0, 33), (130, 300)], 3, 96, 32, FP, False),
    ([(15, 17), (16, 16), (1, 200)], 8, 64, 64, BF, True), ([(5, 1000)], 2, 16, 256, FP, True),
])
def test_read8(lens, hk, d, page, dtype, inner):
    g = torch.Generator().manual_seed(d)
    columns = max(-(-(f + n) // page) for f, n in lens)
    pages = columns * len(lens) + 1
    cache = a8.Cache(pages, hk, page, d, g)
    table = torch.randperm(pages, generator=g)[:columns * len(lens)].view(len(lens), columns)
    dev = cache.on(DEV)
    if not inner:
        dev[:2] = [c.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(a8.F8)
                   for c in dev[:2]]
        dev[2:] = [s.permute(2, 0, 1).contiguous().permute(1, 2, 0) for s in dev[2:]]
    layer = moe.PagedAttention(hk, hk, d, page, 4, len(lens), dtype=dtype)
    n = [n for _, n in lens]
    cu = torch.tensor([0] + n, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(DEV)
    first = torch.tensor([f for f, _ in lens], dtype=torch.int32, device=DEV)
    rows = sum(n)
    out = torch.full((rows + 5, hk, d + 8), 7.0, dtype=dtype, device=DEV)
    k, v = layer.read(dev[0], dev[1], table.to(DEV, torch.int32), cu, first, rows + 5,
                      k_scales=dev[2], v_scales=dev[3], k_out=out[..., :d])
    assert layer.check_device_errors() == 0
    for got, half in ((k, "k"), (v, "v")):
        held, row = cache.held(half), 0
        for s, (f, m) in enumerate(lens):
            p = torch.arange(f, f + m)
            want = held[table[s, p // page], :, p % page]
            assert torch.equal(got[row:row + m].cpu(), want.to(dtype))
            row += m
    # rows of no sequence, and what lies beside the rows, stay
    assert bool((out[rows:] == 7).all()) and bool((out[..., d:] == 7).all())


def test_read8_range():
    layer = moe.PagedAttention(1, 1, 32, 16, 4, 4)
    g = torch.Generator().manual_seed(4)
    cache = a8.Cache(3, 1, 16, 32, g)
    dev = cache.on(DEV)
    table = torch.tensor([[0, 3], [-1, 1], [2, 1]], dtype=torch.int32, device=DEV)
    for cu, first, bad in (([0, 20, 40, 50], [0, 0, 0], True), ([0, 8, 8, 40], [0, 0, 0], False),
                           ([0, 0, 0, 33], [0, 0, 0], True), ([0, 0, 0, 4], [0, 0, -1], True),
                           ([0, 0, 0, 4], [0, 0, 30], True), ([0, 4, 2, 9], [0, 0, 0], False)):
        k, v = layer.read(dev[0], dev[1], table, torch.tensor(cu, dtype=torch.int32, device=DEV),
                          torch.tensor(first, dtype=torch.int32, device=DEV), cu[-1],
                          k_scales=dev[2], v_scales=dev[3])
        assert layer.check_device_errors() == (RANGE if bad else 0)
        # (where rows of sequences do not ascend, which rows are whose is not said)
        if cu[1] >= 4 and cu == sorted(cu):
            assert torch.equal(k[:4].cpu(), cache.held("k")[0, :, :4].transpose(0, 1).to(BF))


# ------------------------------------------------------------------ attention
ATTEND = [
    # (new, keys), hq, hk, dim, page, dtype, options
    ([(1, 1)], 4, 1, 128, 16, BF, {}), ([(1, 4096)], 32, 8, 128, 16, BF, {}),
    ([(1, 300), (1, 17), (1, 0), (0, 40), (1, 1000)], 8, 2, 128, 32, FP, {}),
    ([(4, 700), (2, 3), (4, 4)], 16, 4, 64, 16, BF, {}),
    ([(1, 513), (1, 64)], 12, 12, 96, 64, FP, dict(softcap=30.0)),
    ([(2, 900), (1, 129)], 7, 1, 112, 128, BF, dict(slopes=True)),
    ([(1, 2000), (1, 31)], 64, 1, 16, 256, FP, dict(window=100)),
    ([(3, 777)], 5, 5, 80, 16, BF, dict(window=64, sinks=4)),
    ([(130, 130)], 4, 2, 128, 16, BF, {}), ([(200, 333), (1, 50), (37, 37)], 8, 2, 128, 64, FP, {}),
    ([(300, 300), (5, 600)], 4, 4, 64, 16, FP, dict(window=50, sinks=7)),
    ([(257, 500)], 6, 2, 96, 32, BF, dict(softcap=20.0, slopes=True)),
    ([(77, 200), (128, 128)], 3, 1, 32, 128, BF, dict(prefix=[30, 100])),
    ([(150, 2100)], 16, 2, 128, 256, BF, dict(window=700, sinks=130)),
    ([(65, 1000)], 2, 2, 48, 16, FP, dict(softcap=500.0)),
    ([(40, 90), (90, 90)], 14, 2, 80, 16, FP, dict(prefix=[0, 64], window=20, sinks=3)),
]


@pytest.mark.parametrize("lens,hq,hk,d,page,dtype,opt", ATTEND)
@pytest.mark.parametrize("inner", [True, False])
def test_forward8(lens, hq, hk, d, page, dtype, opt, inner):
    b = a8.Batch8(lens, hq, hk, d, page, dtype, heads_inner=inner, **opt)
    layer = moe.PagedAttention(hq, hk, d, page, max(b.tokens, 1), len(lens), dtype=dtype)
    out, lse = b.run(layer)
    assert layer.check_device_errors() == 0
    b.check(out, lse)
    again, lse2 = b.run(layer)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    layer.close()


@pytest.mark.parametrize("lens", [[(1, 900), (1, 400)], [(140, 900)]])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("gains", [((-12, 3), (-12, 13)), ((0, 1), (-24, -20)), ((-3, 1), (9, 12))])
def test_forward8_blocks_of_different_scales(lens, dtype, gains):
    b = a8.Batch8(lens, 8, 2, 128, 16, dtype, gains=gains, scale=0.05)
    layer = moe.PagedAttention(8, 2, 128, 16, b.tokens, len(lens), dtype=dtype)
    out, lse = b.run(layer)
    err = (out.cpu().double() - b.want).abs()
    # scores of sizes up to 2^3 of the plain ones': their fp32 error with them. A result
    # below fp16's normal range is rounded to 2^-25; one above its range is infinite
    # numerators are fp16, or of the type where the keys are brought to 16 bits (560 rows)
    u = ac.ROUND[dtype]
    numerator = u if lens[0][0] > 100 else 2.0 ** -11
    bound = u * b.want.abs() + (numerator + 8e-4) * b.bound + 2.0 ** -24
    fits = b.want.abs() < 60000
    assert bool((err <= bound)[fits].all()), float((err / bound)[fits].max())
    assert bool(((lse.cpu().double() - b.want_lse).abs() <= 8e-4).all())


SINKS = [([(1, 700), (3, 90)], 8, 2, 128, 16, BF, 64, 4), ([(200, 333), (64, 64)], 4, 4, 64, 32, FP, 50, 7),
         ([(1, 30)], 4, 1, 96, 16, FP, 8, 100), ([(128, 500)], 16, 2, 128, 64, BF, 200, 140)]


@pytest.mark.parametrize("lens,hq,hk,d,page,dtype,window,sinks", SINKS)
def test_sinks_over_a_16_bit_cache(lens, hq, hk, d, page, dtype, window, sinks):
    b = ac.Batch(lens, hq, hk, d, page, dtype, window=window)
    layer = moe.PagedAttention(hq, hk, d, page, b.tokens, len(lens), dtype=dtype)
    out, lse = b.run(layer, sinks=sinks)
    assert layer.check_device_errors() == 0
    row = 0
    for s, (n, kv) in enumerate(lens):
        ids = b.table[s, :-(-kv // page)].long()
        k, v = (p[ids].transpose(1, 2).reshape(-1, hk, d)[:kv].cpu() for p in (b.k_pages, b.v_pages))
        o, a, want = a8.sequence(b.q[row:row + n].cpu(), k, v, b.scale, window=window, sinks=sinks)
        ac.check_attention(out[row:row + n], lse[row:row + n], o, a, want, dtype)
        row += n
    # without a window nothing changes
    plain = b.run(layer, window=0)
    assert torch.equal(plain[0], b.run(layer, window=0, sinks=sinks)[0])
    with pytest.raises(moe.MoeError):
        b.run(layer, sinks=-1)


def test_forward8_refusals():
    b = a8.Batch8([(2, 40)], 4, 2, 64, 32, BF)
    layer = moe.PagedAttention(4, 2, 64, 32, 8, 2)
    for kw in (dict(k_scales=None), dict(v_scales=None), dict(k_scales=b.k_scales.half()),
               dict(k_scales=b.k_scales[:, :, :1]), dict(v_scales=b.v_scales[:-1]),
               dict(k_scales=b.k_scales[:1].expand_as(b.k_scales)),
               dict(k_scales=b.k_scales.cpu())):
        with pytest.raises(ValueError):
            b.run(layer, **kw)
    for kw in (dict(sinks=-1), dict(window=-1), dict(softcap=-1.0), dict(scale=math.nan)):
        with pytest.raises(moe.MoeError):
            b.run(layer, **kw)
    pages = b.k_pages
    for bad in (pages.float().to(BF), pages[:, :, :16], pages.view(torch.uint8)):
        with pytest.raises(ValueError):
            b.k_pages = bad
            b.run(layer)
    b.k_pages = pages
    odd = moe.PagedAttention(4, 2, 72, 32, 8, 2)     # not a multiple of 16
    codes = torch.zeros(3, 2, 32, 72, dtype=torch.uint8, device=DEV).view(a8.F8)
    ones = torch.ones(3, 2, 2, device=DEV)
    q = torch.zeros(2, 4, 72, dtype=BF, device=DEV)
    with pytest.raises(moe.MoeError):
        odd.forward(q, codes, codes, b.table, b.cu_q, b.kv_len, 2, k_scales=ones, v_scales=ones)
    with pytest.raises(ValueError, match="no_grad"):
        layer.forward(b.q.clone().requires_grad_(), b.k_pages, b.v_pages, b.table, b.cu_q, b.kv_len,
                      2, k_scales=b.k_scales, v_scales=b.v_scales)


def test_forward8_range():
    b = a8.Batch8([(1, 40), (1, 30), (1, 90)], 4, 2, 64, 16, BF)
    layer = moe.PagedAttention(4, 2, 64, 16, 8, 4)
    out, _ = b.run(layer)
    b.table[1, 0] = 1 << 20                       # one page of one sequence
    got, _ = b.run(layer)
    assert layer.check_device_errors() == RANGE
    assert torch.equal(got[0], out[0]) and torch.equal(got[2], out[2])
    b.kv_len[1] = 1 << 28                         # a length beyond its table: left out
    fill = torch.full_like(out, 3.0)
    b.run(layer, out=fill)
    assert layer.check_device_errors() == RANGE
    assert torch.equal(fill[0], out[0]) and torch.equal(fill[2], out[2]) and bool((fill[1] == 3).all())
