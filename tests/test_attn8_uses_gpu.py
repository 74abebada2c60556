"""How include/moe_attn8.h's calls are used: captured and replayed, on other streams,
over many sequences and far pages, one after the other as a decoder layer runs them."""
import math

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


class Steps:
    """Tokens of several sequences appended and attended to, step by step."""

    def __init__(self, hq, hk, d, page, dtype, seqs, room, seed=0, norm=True):
        g = self.g = torch.Generator().manual_seed(seed)
        self.hq, self.hk, self.d, self.page, self.dtype, self.seqs = hq, hk, d, page, dtype, seqs
        self.columns = -(-room // page)
        self.table = torch.randperm(seqs * self.columns, generator=g).view(seqs, self.columns)
        self.cache = a8.Cache(seqs * self.columns, hk, page, d, g, fill=False)
        self.dev = self.cache.on(DEV)
        self.freq = ac.frequencies(d).to(DEV)
        self.w = [(torch.rand(d, generator=g) + 0.5).to(dtype) for _ in range(2)]
        self.norm = moe.HeadNorm(self.w[0].to(DEV), self.w[1].to(DEV)) if norm else None
        self.kv = [0] * seqs
        self.layer = moe.PagedAttention(hq, hk, d, page, 4096, seqs, dtype=dtype)

    def batch(self, counts):
        T = sum(counts)
        qkv = torch.randn(T, self.hq + 2 * self.hk, self.d, generator=self.g).to(self.dtype)
        pos, slots = [], []
        for s, n in enumerate(counts):
            for p in range(self.kv[s], self.kv[s] + n):
                pos.append(p)
                slots.append(int(self.table[s, p // self.page]) * self.page + p % self.page)
            self.kv[s] += n
        cu = torch.tensor([0] + list(counts), dtype=torch.int32).cumsum(0, dtype=torch.int32)
        return dict(qkv=qkv.to(DEV), pos=torch.tensor(pos, dtype=torch.int32, device=DEV),
                    slots=torch.tensor(slots, dtype=torch.int64, device=DEV), cu=cu.to(DEV),
                    kv=torch.tensor(self.kv, dtype=torch.int32, device=DEV),
                    table=self.table.to(DEV, torch.int32), max_q=max(counts))

    def run(self, b, **kw):
        q, k, v = b["qkv"].split([self.hq, self.hk, self.hk], dim=1)
        kp, vp, ks, vs = self.dev
        q = self.layer.append(q, k, v, b["pos"], b["slots"], kp, vp, self.freq,
                              norm=self.norm, k_scales=ks, v_scales=vs)
        return q, self.layer.forward(q, kp, vp, b["table"], b["cu"], b["kv"], b["max_q"],
                                     k_scales=ks, v_scales=vs, return_lse=True, **kw)

    def check(self, b, q, out, lse, window=0, sinks=0):
        """The attention over what the cache holds now, whatever it was given."""
        held = [c.view(torch.uint8).cpu().view(a8.F8).float().double() *
                s.cpu().double().repeat_interleave(16, 2)[..., None]
                for c, s in zip(self.dev[:2], self.dev[2:])]
        row = 0
        cu = b["cu"].tolist()
        for s in range(self.seqs):
            n, kv = cu[s + 1] - cu[s], self.kv[s]
            ids = self.table[s, :-(-kv // self.page)]
            k, v = (h[ids].transpose(1, 2).reshape(-1, self.hk, self.d)[:kv] for h in held)
            o, a, want = a8.sequence(q[row:row + n].cpu(), k, v, self.d ** -0.5, window=window,
                                     sinks=sinks)
            if n:
                ac.check_attention(out[row:row + n], lse[row:row + n], o, a, want, self.dtype)
            row += n


@pytest.mark.parametrize("dtype,d,page", [(BF, 128, 16), (FP, 64, 32)])
def test_a_layer_step_by_step(dtype, d, page):
    s = Steps(8, 2, d, page, dtype, 3, 400)
    for counts, kw in (([150, 33, 1], {}), ([7, 1, 0], {}), ([1, 1, 1], {}), ([1, 1, 1], {}),
                       ([90, 1, 60], dict(window=40, sinks=5)), ([2, 2, 2], dict(window=40, sinks=5))):
        b = s.batch(counts)
        q, (out, lse) = s.run(b, **kw)
        assert s.layer.check_device_errors() == 0
        s.check(b, q, out, lse, **kw)
    # and read back: what attention saw, rounded once
    kp, vp, ks, vs = s.dev
    cu = torch.tensor([0] + s.kv, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(DEV)
    k, v = s.layer.read(kp, vp, s.table.to(DEV, torch.int32), cu,
                        torch.zeros(3, dtype=torch.int32, device=DEV), sum(s.kv), k_scales=ks,
                        v_scales=vs)
    held = kp.view(torch.uint8).cpu().view(a8.F8).float() * ks.cpu().repeat_interleave(16, 2)[..., None]
    ids = s.table[1, :-(-s.kv[1] // page)]
    want = held[ids].transpose(1, 2).reshape(-1, 2, d)[:s.kv[1]].to(dtype)
    assert torch.equal(k[s.kv[0]:s.kv[0] + s.kv[1]].cpu(), want)


def test_captured_steps_replay_with_new_lengths():
    # one graph: append and attention of single tokens, over lengths read on the device;
    # a second one of a chunk, with its own scratch; replayed in turn
    s = Steps(8, 2, 128, 16, BF, 4, 700, seed=1)
    first = s.batch([200, 100, 33, 1])
    s.run(first)
    single, chunk = s.batch([1, 1, 1, 1]), s.batch([120, 200, 64, 130])
    single2, chunk2 = s.batch([1, 1, 1, 1]), s.batch([120, 200, 64, 130])
    s.run(single), s.run(chunk)                   # (warm)
    graphs, outs = [], []
    for b in (single, chunk):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.run(b))
        graphs.append(g)
    kv = list(s.kv)
    for i, (b, new) in enumerate(((single, single2), (chunk, chunk2))):
        for name in ("qkv", "pos", "slots", "kv"):
            b[name].copy_(new[name])
    for step, (g, b, (q, (out, lse))) in enumerate(zip(graphs, (single, chunk), outs)):
        g.replay()
        torch.cuda.synchronize()
        s.kv = b["kv"].tolist()
        s.check(b, q, out, lse)
        kept = out.clone()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, kept)
    s.kv = kv
    assert s.layer.check_device_errors() == 0


def test_gradients_captured_beside_eager_ones():
    T, H, D = 37, 4, 64
    x, dy = (torch.randn(T, H, D, device=DEV).to(BF) for _ in range(2))
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    freq, w = ac.frequencies(D).to(DEV), torch.rand(D, device=DEV)
    norm = moe.HeadNorm(w, w)

    def run():
        return moe.moe_attn_norm_rope_backward(dy, dy, x, x, pos, freq, norm)

    eager = run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = run()
    dy.mul_(2.0)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(captured, run()):
        assert torch.equal(a, b)
    # linear in dy: twice the gradient, exactly
    for a, b in zip(captured, eager):
        assert torch.equal(a.float(), 2 * b.float())


@pytest.mark.parametrize("seqs,new", [(33, 1), (700, 1), (300, 5), (2500, 1)])
def test_many_sequences(seqs, new):
    g = torch.Generator().manual_seed(seqs)
    lens = [(min(new, b), b) for b in torch.randint(0, 60, (seqs,), generator=g).tolist()]
    lens[seqs // 2] = (17, 200) if seqs == 33 else lens[seqs // 2]
    b = a8.Batch8(lens, 2, 1, 32, 16, FP, window=40, sinks=2)
    layer = moe.PagedAttention(2, 1, 32, 16, b.tokens, seqs, dtype=FP)
    out, lse = b.run(layer)
    assert layer.check_device_errors() == 0
    b.check(out, lse)


def test_many_sequences_brought_to_16_bits():
    # more sequences than one pass over their pages keeps, 576 rows each, some empty
    lens = [(9, 9 + i % 40) for i in range(2150)] + [(0, 50)] * 3 + [(90, 411)] * 2
    b = a8.Batch8(lens, 64, 1, 16, 16, BF)
    layer = moe.PagedAttention(64, 1, 16, 16, b.tokens, len(lens))
    n = moe.attention.ctypes.c_size_t()
    batch = moe.attention.moe_attn_batch(None, None, None, b.table.shape[1], b.table.shape[1],
                                         len(lens), b.tokens, b.max_q)
    assert layer._library.moe_attn_forward8_scratch_bytes(layer.handle, batch, n) == 0 and n.value
    out, lse = b.run(layer)
    assert layer.check_device_errors() == 0
    b.check(out, lse)


@pytest.mark.parametrize("rows", ["few", "some", "many"])
def test_far_pages(rows):
    # codes beyond 2^32 bytes and scales beyond 2^31 bytes of their tensors
    page, d, hk = 16, 128, 8
    pages = (1 << 32) // (page * d * hk) + 5000
    codes = torch.zeros(pages * hk * page * d, dtype=torch.uint8, device=DEV).view(a8.F8)
    codes = codes.view(pages, hk, page, d)
    big = torch.zeros(pages, 2050, device=DEV)     # 2050 floats from page to page
    scales = big[:, :hk].unflatten(1, (hk, 1))
    n = {"few": 1, "some": 20, "many": 300}[rows]
    layer = moe.PagedAttention(hk * 2, hk, d, page, 512, 1)
    ids = torch.tensor([pages - 1 - 3 * i for i in range(25)], device=DEV)
    kv = 400
    pos = torch.arange(kv, dtype=torch.int32, device=DEV)
    slots = ids[pos.long() // page] * page + pos.long() % page
    k, v = (torch.randn(kv, hk, d, device=DEV).to(BF) for _ in range(2))
    freq = ac.frequencies(0).to(DEV)
    other = codes.clone()
    oscales = scales.clone()
    sv = torch.empty_strided(scales.shape, scales.stride(), device=DEV).zero_()
    layer.append(None, k, v, pos, slots, codes, other, freq, k_scales=scales, v_scales=sv)
    q = torch.randn(n, hk * 2, d, device=DEV).to(BF)
    table = ids[None].to(torch.int32).contiguous()
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    out, lse = layer.forward(q, codes, other, table, cu, torch.tensor([kv], dtype=torch.int32,
                                                                     device=DEV), n,
                             k_scales=scales, v_scales=sv, return_lse=True)
    assert layer.check_device_errors() == 0
    kq, vq = (a8.quantised(x.cpu())[2] for x in (k, v))
    ac.check_attention(out, lse, *a8.sequence(q.cpu(), kq, vq, d ** -0.5), BF)
    rk, rv = layer.read(codes, other, table, torch.tensor([0, kv], dtype=torch.int32, device=DEV),
                        torch.zeros(1, dtype=torch.int32, device=DEV), kv, k_scales=scales,
                        v_scales=sv)
    assert torch.equal(rk.cpu(), kq.to(BF)) and torch.equal(rv.cpu(), vq.to(BF))
    del oscales


def test_calls_on_a_given_stream():
    b = a8.Batch8([(200, 333), (1, 50)], 8, 2, 64, 16, BF)
    layer = moe.PagedAttention(8, 2, 64, 16, b.tokens, 2)
    want, want_lse = b.run(layer)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = b.run(layer, stream=s)              # without scratch: over codes
    s.synchronize()
    b.check(out, lse)
    given = torch.empty_like(want), torch.empty_like(want_lse)
    b.run(layer, stream=s.cuda_stream, out=given[0], lse=given[1])
    s.synchronize()
    assert torch.equal(given[0], out) and torch.equal(given[1], lse)
    with torch.cuda.stream(s):
        again, _ = b.run(layer)
    s.synchronize()
    assert torch.equal(again, want)
    cu = torch.tensor([0, 20], dtype=torch.int32, device=DEV)
    first = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (b.k_pages, b.v_pages, b.table[:1], cu, first, 20)
    sc = dict(k_scales=b.k_scales, v_scales=b.v_scales)
    k, _ = layer.read(*args, **sc)
    k2, _ = layer.read(*args, stream=s, **sc)
    s.synchronize()
    assert torch.equal(k, k2)
    with pytest.raises(ValueError):
        layer.read(*args, stream=s.cuda_stream, **sc)


def test_rows_behind_the_last_sequence_stay():
    for n in (1, 20, 300):
        b = a8.Batch8([(n, 400)], 4, 2, 64, 16, BF)
        layer = moe.PagedAttention(4, 2, 64, 16, n + 9, 1)
        b.q = torch.cat([b.q, b.q[:1].expand(9, 4, 64)])
        out = torch.full_like(b.q, 5.0)
        lse = torch.full((n + 9, 4), 5.0, device=DEV)
        b.run(layer, out=out, lse=lse)
        b.check(out[:n], lse[:n])
        assert bool((out[n:] == 5).all()) and bool((lse[n:] == 5).all())


def test_masks_that_leave_nothing():
    # new tokens without keys (a length of zero is refused by range, none is not)
    b = a8.Batch8([(1, 1), (0, 0), (1, 40)], 4, 2, 64, 16, BF)
    b.kv_len[0] = 0                                # its query stands before key 0
    layer = moe.PagedAttention(4, 2, 64, 16, 8, 4)
    out, lse = b.run(layer)
    assert not out[0].any() and bool((lse[0] == -math.inf).all())
    assert layer.check_device_errors() == 0
    ac.check_attention(out[1:], lse[1:], b.want[1:], b.bound[1:], b.want_lse[1:], BF)


def test_expanded_weights_are_refused():
    # a gradient of their shape would have rows that no head has
    x = torch.zeros(2, 3, 64, dtype=BF, device=DEV)
    pos, freq = torch.zeros(2, dtype=torch.int32, device=DEV), ac.frequencies(64).to(DEV)
    w = torch.ones(64, dtype=BF, device=DEV)
    for call in (lambda n: moe.moe_attn_norm_rope(x, None, pos, freq, n),
                 lambda n: moe.moe_attn_norm_rope_backward(x, None, x, None, pos, freq, n)):
        with pytest.raises(ValueError, match="q_weight"):
            call(moe.HeadNorm(w.expand(3, 64), None))
    shapes = [t.shape for t in moe.moe_attn_norm_rope_backward(
        x[:, :1], None, x[:, :1], None, pos, freq, moe.HeadNorm(w[None], None)) if t is not None]
    assert shapes == [(2, 1, 64), (1, 64)]


def test_read8_of_too_many_rows_is_refused():
    layer = moe.PagedAttention(1, 1, 16, 16, 8, 2)
    c = moe.attention
    byte = torch.zeros(1024, device=DEV)
    at = byte.data_ptr()
    rows = c.moe_attn_rows(at, 16, 16)
    cache = c.moe_attn_cache8(at, at, at, at, 1, 256, 16, 256, 0, 0, 0)
    for n, status in ((2**30 + 1, -3), (2**31 - 1, -3), (-1, -1)):  # too many, invalid
        extent = c.moe_attn_extent(at, at, at, 1, 1, 1, n)
        assert layer._library.moe_attn_read8(layer.handle, cache, extent, rows, rows, None) == status


def test_no_room_to_bring_keys_to_16_bits():
    # torch has no memory for it: the call goes on without
    b = a8.Batch8([(300, 4000)] * 3, 8, 2, 128, 64, BF)
    layer = moe.PagedAttention(8, 2, 128, 64, b.tokens, 3)
    out, lse = torch.empty_like(b.q), torch.empty(b.tokens, 8, device=DEV)
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 20)) / total)
    try:
        b.run(layer, out=out, lse=lse)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert layer.check_device_errors() == 0
    b.check(out, lse)
