"""GPU tests of attention over many sequences and many entries: more than one of
either for every thread that divides the work, sequences read again where they are
too many to be kept, empty ones among them. Against the definitions in fp64."""
import random

import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn_cases as ac

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16


def _lens(count, most_new, seed):
    rng = random.Random(seed)
    lens = []
    for _ in range(count):
        n = min(most_new, rng.choice([0, 0, 1, 1, 2, 17, most_new, rng.randint(0, most_new)]))
        lens.append((n, rng.choice([n, n + rng.randint(0, 30), n // 2, 0, n + 140])))
    return lens


@pytest.mark.parametrize("count,most_new,hq,hk,d,page,dtype,kw", [
    (385, 40, 4, 2, 16, 16, BF, {}),            # one more than the threads that divide
    (500, 40, 4, 2, 64, 16, BF, {}),
    (1200, 70, 6, 3, 72, 32, FP, dict(window=20)),
    (4096, 40, 2, 1, 16, 16, BF, dict(slopes=True)),
    (4097, 40, 2, 1, 16, 16, FP, {}),           # one more than are kept
    (5000, 40, 2, 2, 8, 16, BF, dict(softcap=10.0)),
    (16384, 9, 2, 1, 8, 16, BF, {}),            # as many as a handle takes
    (700, 150, 16, 1, 16, 64, FP, {}),          # several entries a sequence
    (500, 4, 4, 1, 64, 16, BF, {}),             # the few-token kernel
    (5000, 2, 8, 1, 16, 16, FP, dict(window=9)),
    (16384, 1, 2, 1, 8, 32, BF, {}),
])
def test_many_sequences(count, most_new, hq, hk, d, page, dtype, kw):
    lens = _lens(count, most_new, count)
    lens[0] = lens[-1] = (0, 3)
    lens[count // 2] = (most_new, most_new + 5)
    b = ac.Batch(lens, hq, hk, d, page, dtype, **kw)
    assert b.max_q == most_new
    layer = moe.PagedAttention(hq, hk, d, page, b.tokens, count, dtype=dtype)
    out, lse = b.run(layer)
    b.check(out, lse)
    for _ in range(2):
        o2, l2 = b.run(layer)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    assert layer.check_device_errors() == 0


@pytest.mark.parametrize("n,before,kw", [(2100, 0, {}), (3001, 500, dict(window=700)),
                                         (1700, 90, dict(softcap=30.0))])
def test_many_entries_of_one_prompt(n, before, kw):
    # 64 query heads on a kv head: two tokens a tile, four an entry
    hq, hk, d, page, dtype = 64, 1, 32, 64, BF
    g = torch.Generator().manual_seed(n)
    kv = n + before
    used = -(-kv // page)
    q = torch.randn(n, hq, d, generator=g).to(dtype)
    kp = torch.randn(used, hk, page, d, generator=g).to(dtype)
    vp = torch.randn(used, hk, page, d, generator=g).to(dtype)
    i32 = dict(dtype=torch.int32, device=DEV)
    layer = moe.PagedAttention(hq, hk, d, page, n, 1, dtype=dtype)
    out, lse = layer.forward(q.to(DEV), kp.to(DEV), vp.to(DEV), torch.arange(used, **i32)[None],
                             torch.tensor([0, n], **i32), torch.tensor([kv], **i32), n,
                             return_lse=True, **kw)
    k, v = (t.transpose(1, 2).reshape(-1, hk, d) for t in (kp, vp))
    for a in range(0, n, 150):
        z = min(n, a + 150)
        want, bound, want_lse = ac.sequence(q[a:z], k[:before + z], v[:before + z], d ** -0.5, **kw)
        ac.check_attention(out[a:z], lse[a:z], want, bound, want_lse, dtype)
    assert layer.check_device_errors() == 0


def test_a_bad_length_among_many_leaves_one_sequence_out():
    lens = [(1 + i % 33, 40 + i % 50) for i in range(4500)]
    b = ac.Batch(lens, 2, 1, 8, 16, BF)
    layer = moe.PagedAttention(2, 1, 8, 16, b.tokens, len(lens))
    out, lse = b.run(layer)
    b.check(out, lse)
    b.kv_len[3000] = 10 ** 6
    a, z = int(b.cu_q[3000]), int(b.cu_q[3001])
    o2, l2 = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    b.run(layer, out=o2, lse=l2)
    assert layer.check_device_errors() == 0x2
    assert bool((o2[a:z] == 7.0).all()) and bool((l2[a:z] == 7.0).all())
    o2[a:z], l2[a:z] = out[a:z], lse[a:z]
    b.check(o2, l2)
