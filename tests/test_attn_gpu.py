"""GPU tests of the attention operators (include/moe_attn.h) against their
definitions in fp64 (attn_cases.py, which derives the bounds)."""
import math

import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn_cases as ac

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.lib()


# ------------------------------------------------------------------ rotary positions
@pytest.mark.parametrize("tokens,heads,dim,rot,layout,dtype", [
    (1, 40, 128, 128, "half", BF), (7, 3, 128, 64, "interleaved", FP),
    (65, 5, 96, 24, "half", BF), (33, 1, 80, 40, "half", FP), (5, 2, 256, 256, "half", BF),
    (4, 9, 256, 256, "interleaved", FP), (3, 2, 6, 2, "half", BF), (3, 2, 5, 4, "interleaved", FP),
    (9, 3, 64, 0, "half", BF), (301, 2, 64, 64, "interleaved", BF), (2, 300, 8, 8, "half", FP),
    (2, 1, 255, 254, "half", BF), (2, 1, 255, 254, "interleaved", BF),
])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(tokens, heads, dim, rot, layout, dtype, inverse):
    g = torch.Generator().manual_seed(tokens + dim)
    x = torch.randn(tokens, heads, dim, generator=g).to(dtype)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (tokens,), generator=g).to(torch.int32)
    pos[0] = 3
    freq = ac.frequencies(rot)
    want, slack = ac.rotary(x, pos, freq, layout, 1.25, inverse)
    got = moe.moe_attn_rope(x.to(DEV), pos.to(DEV), freq.to(DEV), layout=layout, magnitude=1.25,
                            inverse=inverse)
    ac.check_rotary(got, want, slack, dtype)
    assert torch.equal(got[..., rot:].cpu(), x[..., rot:])


@pytest.mark.parametrize("offset,pad", [(0, 0), (4, 4), (1, 3), (8, 8), (2, 6)])
def test_rope_strided_in_place(offset, pad):
    # a slice of a fused buffer at any alignment, turned in place; what lies
    # beside it stays
    T, H, D = 19, 4, 64
    buf = torch.randn(T, H * (D + pad) + offset, device=DEV).to(BF)
    view = torch.as_strided(buf, (T, H, D), (buf.stride(0), D + pad, 1), offset)
    before, x = buf.clone(), view.clone()
    pos = torch.arange(100, 100 + T, dtype=torch.int32, device=DEV)
    freq = ac.frequencies(D)
    want, slack = ac.rotary(x, pos, freq, "half")
    got = moe.moe_attn_rope(view, pos, freq.to(DEV), out=view)
    assert got.data_ptr() == view.data_ptr()
    ac.check_rotary(view, want, slack, BF)
    touched = torch.zeros(buf.numel(), dtype=torch.bool, device=DEV)
    torch.as_strided(touched, (T, H, D), (buf.stride(0), D + pad, 1), offset).fill_(True)
    assert torch.equal(buf.flatten()[~touched], before.flatten()[~touched])


def test_rope_gradient_against_differences_and_transpose():
    # the map is linear: <g, rope(dx)> == <inverse(g), dx>; and inverse undoes
    # it up to the square of the magnitude
    T, H, D = 6, 3, 64
    pos = torch.randint(0, 1 << 20, (T,), device=DEV).to(torch.int32)
    freq = ac.frequencies(D).to(DEV)
    x = torch.randn(T, H, D, device=DEV).to(FP)
    g = torch.randn(T, H, D, device=DEV).to(FP)
    for layout in ("half", "interleaved"):
        y = moe.moe_attn_rope(x, pos, freq, layout=layout, magnitude=1.5)
        gx = moe.moe_attn_rope(g, pos, freq, layout=layout, magnitude=1.5, inverse=True)
        # each entry of y and gx is rounded once (2^-11) from fp32 angles and products
        u = 2.0 ** -11 + 2.0 ** -18
        lhs, rhs = g.double() * y.double(), gx.double() * x.double()
        bound = u * float(lhs.abs().sum() + rhs.abs().sum())
        assert abs(float(lhs.sum() - rhs.sum())) <= bound
        # central differences of L = <g, rope(x)> in single coordinates, step 1
        for (t, h, i) in ((0, 0, 0), (3, 1, 17), (5, 2, 63)):
            e = torch.zeros_like(x)
            e[t, h, i] = 1.0
            d = (g.double() * moe.moe_attn_rope(e, pos, freq, layout=layout,
                                                magnitude=1.5).double()).sum()
            # at most two entries of the column, each rounded once
            assert abs(float(d) - float(gx[t, h, i])) <= 2.0 ** -11 * 1.5 * 4 * float(
                g[t, h].double().abs().max()) + 2.0 ** -11 * abs(float(d))


def test_rope_empty_and_other_stream():
    freq = ac.frequencies(64).to(DEV)
    e = torch.empty(0, 4, 64, dtype=BF, device=DEV)
    pos0 = torch.empty(0, dtype=torch.int32, device=DEV)
    assert moe.moe_attn_rope(e, pos0, freq).shape == (0, 4, 64)
    x = torch.randn(50, 4, 64, device=DEV).to(BF)
    pos = torch.arange(50, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.moe_attn_rope(x, pos, freq, stream=s)
    s.synchronize()
    want, slack = ac.rotary(x, pos, freq.cpu(), "half")
    ac.check_rotary(got, want, slack, BF)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("tokens,hq,hk,dim,rot,page,layout,dtype,inner", [
    (1, 4, 1, 128, 128, 16, "half", BF, True), (64, 32, 8, 128, 128, 16, "half", BF, False),
    (77, 6, 2, 80, 40, 32, "half", FP, True), (130, 7, 7, 96, 24, 64, "interleaved", BF, False),
    (17, 64, 1, 8, 8, 256, "interleaved", FP, True), (33, 4, 4, 64, 0, 128, "half", BF, True),
])
@pytest.mark.parametrize("with_q", [True, False])
def test_append(tokens, hq, hk, dim, rot, page, layout, dtype, inner, with_q):
    g = torch.Generator().manual_seed(tokens)
    pages = tokens // page + 5
    shape = (pages, hk, page, dim) if inner else (pages, page, hk, dim)
    kp = torch.randn(shape, generator=g).to(dtype).to(DEV)
    vp = torch.randn(shape, generator=g).to(dtype).to(DEV)
    if not inner:
        kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
    qkv = torch.randn(tokens, hq + 2 * hk, dim, generator=g).to(dtype)
    dq = qkv.to(DEV)
    q, k, v = dq[:, :hq], dq[:, hq:hq + hk], dq[:, hq + hk:]
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    slots[tokens // 3] = -1 if tokens > 1 else slots[0]
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g).to(torch.int32)
    freq = ac.frequencies(rot)
    layer = moe.PagedAttention(hq, hk, dim, page, tokens, 1, dtype=dtype)
    k0, v0 = kp.clone(), vp.clone()
    out = layer.append(q if with_q else None, k, v, pos.to(DEV), slots.to(DEV), kp, vp,
                       freq.to(DEV), layout=layout, magnitude=0.75)
    if with_q:
        want, slack = ac.rotary(qkv[:, :hq], pos, freq, layout, 0.75)
        ac.check_rotary(out, want, slack, dtype)
    else:
        assert out is None
    want, slack = ac.rotary(qkv[:, hq:hq + hk], pos, freq, layout, 0.75)
    keep = torch.ones(pages * page, dtype=torch.bool)
    for t, slot in enumerate(slots.tolist()):
        if slot < 0:
            continue
        keep[slot] = False
        ac.check_rotary(kp[slot // page, :, slot % page], want[t], slack[t], dtype)
        assert torch.equal(vp[slot // page, :, slot % page], v[t])
    keep = keep.view(pages, page).to(DEV)
    for now, was in ((kp, k0), (vp, v0)):
        assert torch.equal(now.transpose(1, 2)[keep], was.transpose(1, 2)[keep])
    assert layer.check_device_errors() == 0


def test_append_reports_a_slot_past_the_cache():
    layer = moe.PagedAttention(4, 2, 64, 16, 8, 1)
    kp = torch.zeros(2, 2, 16, 64, dtype=BF, device=DEV)
    vp = torch.zeros_like(kp)
    k = torch.ones(3, 2, 64, dtype=BF, device=DEV)
    slots = torch.tensor([0, 32, 31], dtype=torch.int64, device=DEV)
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)
    layer.append(None, k, k, pos, slots, kp, vp, ac.frequencies(64).to(DEV))
    assert layer.check_device_errors() == 0x2
    assert layer.check_device_errors() == 0
    assert float(vp.sum()) == 2 * 2 * 64  # slots 0 and 31 written, the other left out


# ------------------------------------------------------------------ attention
SHAPES = [  # hq, hk, d, page, dtype
    (32, 8, 128, 16, BF), (4, 4, 64, 64, FP), (6, 2, 96, 32, BF), (7, 1, 80, 128, FP),
    (16, 2, 128, 256, FP), (64, 1, 64, 16, BF), (2, 2, 8, 16, FP), (5, 1, 120, 32, BF),
]
DECODE = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 63), (1, 64), (1, 65), (1, 127),
          (1, 128), (1, 129), (1, 1000)]
MIXED = [(1, 700), (130, 130), (3, 3), (1, 1), (64, 300), (257, 511), (17, 40), (2, 2000)]


def _layer(b, shape, tokens=None):
    hq, hk, d, page, dtype = shape
    return moe.PagedAttention(hq, hk, d, page, tokens or b.tokens, len(b.lens), dtype=dtype)


def _check(lens, shape, **kw):
    b = ac.Batch(lens, *shape, **kw)
    layer = _layer(b, shape)
    out, lse = b.run(layer)
    b.check(out, lse)
    assert layer.check_device_errors() == 0
    return b, layer, out, lse


@pytest.mark.parametrize("shape", SHAPES)
def test_single_tokens(shape):
    _check(DECODE, shape)


@pytest.mark.parametrize("shape", SHAPES)
def test_mixed_lengths(shape):
    _check(MIXED, shape)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kw", [
    dict(softcap=20.0), dict(window=1), dict(window=100), dict(slopes=True),
    dict(prefix=[0, 130, 2, 1, 200, 400, 5000, -3]),
    dict(softcap=5.0, window=70, slopes=True, prefix=[3, 0, 0, 9, 20, 300, 17, 130]),
])
def test_scores_and_masks(shape, kw):
    _check(MIXED, shape, **kw)


@pytest.mark.parametrize("shape", SHAPES[:4])
@pytest.mark.parametrize("kw", [dict(), dict(window=40), dict(prefix=[8] * 12, window=33)])
def test_few_tokens(shape, kw):
    lens = [(2, 2), (3, 90), (4, 64), (5, 129), (2, 1), (4, 2), (1, 0), (3, 0), (8, 8), (16, 700),
            (6, 333), (2, 128)]
    _check(lens, shape, **kw)


@pytest.mark.parametrize("shape", SHAPES[:4])
def test_rows_without_keys(shape):
    # more new tokens than keys: the first rows see nothing, and no keys at all
    _check([(40, 17), (300, 129), (1, 0), (5, 0), (200, 0), (129, 128)], shape)


def test_empty_sequences_and_unlisted_rows():
    shape = (8, 2, 64, 16, BF)
    b = ac.Batch([(0, 5), (3, 9), (0, 0), (140, 200), (0, 64)], *shape)
    layer = moe.PagedAttention(8, 2, 64, 16, b.tokens + 7, 8, dtype=BF)
    q = torch.cat([b.q, torch.full((7, 8, 64), math.nan, dtype=BF, device=DEV)])
    out = torch.full_like(q, 7.0)
    lse = torch.full((b.tokens + 7, 8), 5.0, device=DEV)
    layer.forward(q, b.k_pages, b.v_pages, b.table, b.cu_q, b.kv_len, 200, out=out, lse=lse)
    b.check(out[:b.tokens], lse[:b.tokens])
    assert bool((out[b.tokens:] == 7.0).all()) and bool((lse[b.tokens:] == 5.0).all())


@pytest.mark.parametrize("lens", [MIXED, DECODE])
def test_strides_and_cache_orders(lens):
    shape = (12, 4, 64, 32, BF)
    b = ac.Batch(lens, *shape, heads_inner=False)
    layer = _layer(b, shape)
    wide = torch.full((b.tokens, 12 + 8, 64), 3.0, dtype=BF, device=DEV)
    wide[:, 4:16] = b.q
    dst = torch.full((b.tokens, 12, 72), 9.0, dtype=BF, device=DEV)
    q, out = wide[:, 4:16], dst[..., :64]
    layer.forward(q, b.k_pages, b.v_pages, b.table, b.cu_q, b.kv_len, b.max_q, out=out)
    b.check(out, None)
    assert bool((dst[..., 64:] == 9.0).all())
    # heads outside tokens
    q2 = b.q.transpose(0, 1).contiguous().transpose(0, 1)
    o2 = torch.empty(12, b.tokens, 64, dtype=BF, device=DEV).transpose(0, 1)
    layer.forward(q2, b.k_pages, b.v_pages, b.table, b.cu_q, b.kv_len, b.max_q, out=o2)
    assert torch.equal(o2, out)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("order", ["heads", "tokens", "padded", "one page"])
def test_cache_orders_of_wide_heads(page, order):
    # heads of 128 values come in other boxes where the cache is regular
    lens, hk = [(150, 16)] if order == "one page" else MIXED + [(150, 513)], 2
    shape = (8, hk, 128, page, BF)
    b = ac.Batch(lens, *shape, heads_inner=order != "tokens")
    if order == "one page":   # a cache of a single page
        first = b.table[0, 0].item()
        b.k_pages, b.v_pages = b.k_pages[first:first + 1], b.v_pages[first:first + 1]
        b.table = torch.zeros_like(b.table)
    if order == "padded":
        for name in ("k_pages", "v_pages"):
            t = getattr(b, name)
            wide = torch.full((t.shape[0], hk + 1, page, 128), math.nan, dtype=BF, device=DEV)
            wide[:, :hk] = t
            setattr(b, name, wide[:, :hk])
    layer = _layer(b, shape)
    b.check(*b.run(layer))
    assert layer.check_device_errors() == 0


def test_runs_are_identical_and_handles_are_reused():
    shape = (32, 8, 128, 16, BF)
    b = ac.Batch(MIXED, *shape)
    layer = _layer(b, shape, tokens=1000)
    out, lse = b.run(layer)
    small = ac.Batch([(1, 3000), (1, 77)], *shape, seed=5)
    for _ in range(3):
        small.check(*small.run(layer))
        o2, l2 = b.run(layer)
        assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("kw", [dict(softcap=30.0), dict(softcap=3.0, window=40), dict(slopes=True),
                                dict(prefix=[70] * 40)])
def test_what_does_not_exist_changes_nothing(kw):
    # rows behind a tile's tokens and keys behind a sequence's end hold what was
    # there before: runs after other work repeat bit by bit
    shape = (15, 5, 40, 64, BF)
    lens = [(1 + 7 * i % 90, 1 + 37 * i % 200) for i in range(40)]
    b = ac.Batch(lens, *shape, **kw)
    layer = _layer(b, shape, tokens=4000)
    out, lse = b.run(layer)
    b.check(out, lse)
    others = [ac.Batch([(300, 700), (90, 90), (200, 10)], *shape, seed=i) for i in (1, 2)]
    for i in range(6):
        others[i % 2].q.mul_(1 + i)
        others[i % 2].run(layer)
        o2, l2 = b.run(layer)
        assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("d,page", [(128, 64), (64, 16)])
def test_many_blocks_per_processor(d, page):
    # some 60 blocks of keys for every SM: each ring of stages goes round many
    # times, and a run repeats the one before bit by bit
    shape = (8, 8, d, page, BF)
    b = ac.Batch([(1, 18000), (1, 16384), (1, 17011), (1, 16001)], *shape)
    layer = _layer(b, shape)
    out, lse = b.run(layer)
    b.check(out, lse)
    for _ in range(20):
        o2, l2 = b.run(layer)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    assert layer.check_device_errors() == 0


@pytest.mark.parametrize("hq,hk,d,page,lens,kw", [
    (8, 8, 64, 64, [(1500, 30000)], dict()),
    (32, 8, 128, 16, [(300, 65536), (1, 40000)], dict()),
    (16, 4, 96, 32, [(200, 50000), (64, 33333), (130, 60001)], dict(softcap=20.0)),
    (8, 8, 64, 128, [(700, 40000), (700, 40000)], dict(window=20000)),
    (4, 1, 128, 64, [(40, 300000), (200, 200000)], dict()),
    (8, 8, 128, 64, [(1500, 30000)], dict()),
    (16, 4, 96, 32, [(200, 50000), (64, 33333), (130, 60001)], dict()),
    (8, 8, 128, 128, [(700, 40000), (700, 40000)], dict(window=20000)),
    (32, 8, 128, 16, [(1000, 65536)], dict()),
    (8, 1, 128, 64, [(16, 400000), (3, 5), (31, 17)], dict()),
])
def test_long_caches_against_single_tokens(hq, hk, d, page, lens, kw):
    # few items over many keys: their cuts and joins, against every query as a
    # sequence of its own (the few-token kernel), both within the bound of
    # attn_cases.py of the definition, with A from a run on |V|
    g = torch.Generator(device=DEV).manual_seed(7)
    used = [-(-kv // page) for _, kv in lens]
    shape = (sum(used), hk, page, d)
    kp = torch.randn(shape, generator=g, device=DEV).to(BF)
    vp = torch.randn(shape, generator=g, device=DEV).to(BF)
    n, kv = [a for a, _ in lens], [b for _, b in lens]
    T = sum(n)
    q = torch.randn(T, hq, d, generator=g, device=DEV).to(BF)
    order = torch.randperm(sum(used), generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(len(lens), max(used), dtype=torch.int32, device=DEV)
    for s, (u, part) in enumerate(zip(used, order.split(used))):
        table[s, :u] = part
    i32 = dict(dtype=torch.int32, device=DEV)
    cu = torch.tensor([0] + n).cumsum(0).to(**i32)
    layer = moe.PagedAttention(hq, hk, d, page, T, max(T, 1))
    out, lse = layer.forward(q, kp, vp, table, cu, torch.tensor(kv, **i32), max(n),
                             return_lse=True, **kw)
    rows = torch.cat([torch.full((a,), s) for s, a in enumerate(n)]).to(DEV)
    # a row in front of the first key sees none
    ends = torch.cat([torch.arange(b - a + 1, b + 1) for a, b in lens]).clamp(min=0).to(**i32)
    each = dict(page_table=table[rows], cu_q=torch.arange(T + 1, **i32), kv_len=ends, max_q=1)
    one, lse1 = layer.forward(q, kp, vp, return_lse=True, **each, **kw)
    a = layer.forward(q, kp, vp.abs(), **each, **kw).double()
    u = ac.ROUND[BF]
    bound = 2 * (u * one.double().abs() + (u + 1e-4) * a * (1 + 2 * u)) + 2.0 ** -23
    diff = out.double() - one.double()
    assert bool((diff.abs() <= bound).all())
    # of independent values, with numerators and outputs rounded once in either
    # run, the whole differs by at most sqrt(4 u^2 / 3) of its norm, here 2 u
    assert float(diff.norm() / one.double().norm()) <= 2 * u
    assert bool(((lse == lse1) | ((lse - lse1).abs() <= 2e-4 + 2.0 ** -21 * lse1.abs())).all())
    for _ in range(3):
        o2, l2 = layer.forward(q, kp, vp, table, cu, torch.tensor(kv, **i32), max(n),
                               return_lse=True, **kw)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    assert layer.check_device_errors() == 0


def test_graph_replays_with_new_lengths():
    shape = (8, 2, 128, 16, BF)
    lens = [[(1, 400), (120, 300), (1, 9)], [(1, 33), (120, 128), (1, 390)]]
    bs = [ac.Batch(x, *shape, seed=i) for i, x in enumerate(lens)]
    layer = _layer(bs[0], shape)
    cols = max(b.table.shape[1] for b in bs)
    pages = max(b.k_pages.shape[0] for b in bs)
    table = torch.zeros(3, cols, dtype=torch.int32, device=DEV)
    kp = torch.full((pages, 2, 16, 128), math.nan, dtype=BF, device=DEV)
    vp, q = kp.clone(), torch.empty_like(bs[0].q)
    kv, out = bs[0].kv_len.clone(), torch.empty_like(bs[0].q)

    def fill(b):
        table[:, :b.table.shape[1]] = b.table
        kp[:b.k_pages.shape[0]], vp[:b.k_pages.shape[0]] = b.k_pages, b.v_pages
        q.copy_(b.q)
        kv.copy_(b.kv_len)

    def call():
        layer.forward(q, kp, vp, table, bs[0].cu_q, kv, 120, out=out)

    fill(bs[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for b in (bs[1], bs[0], bs[1]):
        fill(b)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        b.check(out, None)


@pytest.mark.parametrize("n", [1, 150])
def test_offsets_past_32_bits(n):
    # pages 2^31 elements apart: byte offsets past 2^33
    hq, hk, d, page, kv = 8, 2, 64, 16, 200
    b = ac.Batch([(n, kv)], hq, hk, d, page, BF)
    used = -(-kv // page)
    free = torch.cuda.mem_get_info()[0]
    stride = 2 ** 31 + 4096
    if free < (2 * (used + 1) * stride + (1 << 30)):
        pytest.skip("needs more free device memory")
    big = torch.empty((used + 1) * stride, dtype=BF, device=DEV)
    block = hk * page * d
    shape, strides = (used, hk, page, d), (stride, page * d, d, 1)
    kp, vp = big.as_strided(shape, strides, 0), big.as_strided(shape, strides, block)
    ids = b.table[0, :used].long()
    kp.copy_(b.k_pages[ids])
    vp.copy_(b.v_pages[ids])
    b.table = torch.arange(used, dtype=torch.int32, device=DEV)[None]
    b.k_pages, b.v_pages = kp, vp
    layer = moe.PagedAttention(hq, hk, d, page, n, 1)
    b.check(*b.run(layer))
    # the append's slots reach the far pages too
    slots = torch.tensor([used * page - 1], dtype=torch.int64, device=DEV)
    row = torch.randn(1, hk, d, device=DEV).to(BF)
    layer.append(None, row, row, torch.zeros(1, dtype=torch.int32, device=DEV), slots, kp, vp,
                 ac.frequencies(d).to(DEV))
    assert torch.equal(vp[used - 1, :, page - 1], row[0])
    assert torch.equal(kp[used - 1, :, page - 1], row[0])
    assert layer.check_device_errors() == 0


@pytest.mark.parametrize("n", [1, 140])
def test_device_checks_report(n):
    shape = (8, 2, 64, 16, BF)
    b = ac.Batch([(n, 300), (n, 200)], *shape)
    layer = _layer(b, shape)
    out, lse = b.run(layer)
    good = b.table.clone()
    for bad in (-1, b.k_pages.shape[0], 2 ** 31 - 1):  # page ids outside the cache
        b.table = good.clone()
        b.table[0, 3] = bad
        o2, l2 = b.run(layer)
        assert layer.check_device_errors() == 0x2
        assert torch.equal(o2[n:], out[n:]) and torch.equal(l2[n:], lse[n:])
    b.table = good
    kv = b.kv_len
    for bad in (-5, (good.shape[1] + 1) * 16):          # lengths outside the table
        b.kv_len = torch.tensor([bad, 200], dtype=torch.int32, device=DEV)
        o2, l2 = b.run(layer)
        assert layer.check_device_errors() == 0x2
        assert torch.equal(o2[n:], out[n:]) and torch.equal(l2[n:], lse[n:])
    b.kv_len = kv
    cu = b.cu_q
    for bad in ([0, n, 10 ** 6], [0, -1, 2 * n], [5 * n, n, 2 * n]):  # rows outside q
        b.cu_q = torch.tensor(bad, dtype=torch.int32, device=DEV)
        b.run(layer)
        assert layer.check_device_errors() == 0x2
    b.cu_q = cu
    o2, l2 = b.run(layer)
    assert torch.equal(o2, out) and layer.check_device_errors() == 0


def test_non_finite_scores():
    # an infinite score takes its row to NaN or onto one key, and no other row
    shape = (4, 4, 64, 16, BF)
    for lens in ([(1, 200), (1, 200)], [(130, 200), (3, 200)]):
        b = ac.Batch(lens, *shape)
        layer = _layer(b, shape)
        out, _ = b.run(layer)
        b.q[0, 1] = math.nan
        o2, _ = b.run(layer)
        assert bool(o2[0, 1].isnan().all())
        o2[0, 1] = out[0, 1]
        assert torch.equal(o2, out)


def test_large_scores_do_not_overflow():
    shape = (4, 2, 64, 16, BF)
    _check([(1, 300), (150, 300)], shape, scale=60.0)


def test_refusals():
    layer = moe.PagedAttention(8, 2, 64, 16, 32, 4)
    b = ac.Batch([(3, 40), (2, 20)], 8, 2, 64, 16, BF)
    ok = dict(q=b.q, k_pages=b.k_pages, v_pages=b.v_pages, page_table=b.table, cu_q=b.cu_q,
              kv_len=b.kv_len, max_q=3)
    layer.forward(**ok)
    bad = [
        dict(q=b.q.to(FP)), dict(q=b.q[:, :4]), dict(q=b.q.cpu()),
        dict(q=b.q.transpose(1, 2).contiguous().transpose(1, 2)),
        dict(k_pages=b.k_pages[:, :, :8]), dict(v_pages=b.v_pages.to(FP)),
        dict(v_pages=b.v_pages[:, :1]), dict(page_table=b.table.long()),
        dict(page_table=b.table[:1]), dict(cu_q=b.cu_q[:2]), dict(cu_q=b.cu_q.long()),
        dict(kv_len=b.kv_len.cpu()), dict(slopes=torch.ones(3, device=DEV)),
        dict(prefix=torch.ones(2, device=DEV)), dict(out=torch.empty_like(b.q)[:4]),
        dict(lse=torch.empty(5, 8, device=DEV, dtype=torch.float64)),
    ]
    for kw in bad:
        with pytest.raises(ValueError):
            layer.forward(**{**ok, **kw})
    wide = torch.zeros(5, 8, 65, dtype=BF, device=DEV)
    many = torch.zeros(40, 8, 64, dtype=BF, device=DEV)
    for kw, status in [(dict(softcap=-1.0), -1), (dict(softcap=math.inf), -1),
                       (dict(window=-1), -1), (dict(scale=math.nan), -1), (dict(max_q=-1), -1),
                       (dict(out=b.q), -1), (dict(q=wide[..., :64]), -4), (dict(q=many), -3)]:
        with pytest.raises(moe.MoeError) as e:
            layer.forward(**{**ok, **kw})
        assert e.value.status == status, kw
    freq = ac.frequencies(64).to(DEV)
    k = torch.zeros(5, 2, 64, dtype=BF, device=DEV)
    pos = torch.zeros(5, dtype=torch.int32, device=DEV)
    slots = torch.arange(5, device=DEV)
    base = dict(q=b.q, k=k, v=k, positions=pos, slots=slots, k_pages=b.k_pages,
                v_pages=b.v_pages, freq=freq)
    for kw in [dict(k=k[:4]), dict(v=k.to(FP)), dict(slots=slots.to(torch.int32)),
               dict(positions=slots), dict(freq=freq.float()), dict(layout="other"),
               dict(q=b.q[:3]), dict(q=None, q_out=b.q)]:
        with pytest.raises(ValueError):
            layer.append(**{**base, **kw})
    with pytest.raises(moe.MoeError):
        layer.append(**{**base, "freq": ac.frequencies(128).to(DEV)})
    with pytest.raises(moe.MoeError):
        moe.moe_attn_rope(b.q, pos, freq, magnitude=math.inf)
    with pytest.raises(moe.MoeError):  # overlaps its input, shifted
        big = torch.zeros(6, 8, 64, dtype=BF, device=DEV)
        moe.moe_attn_rope(big[:5], pos, freq, out=big[1:])
    with pytest.raises(ValueError):
        moe.moe_attn_rope(b.q.float(), pos, freq)
