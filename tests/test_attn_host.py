"""Host-side checks of the attention operators: names, refusals before any
device work, the rotary frequencies and the cache's bookkeeping. No kernel is
launched here."""
import ctypes
import math
import os
import re

import pytest

import w4a16_routed_expert_router_gb300 as moe
from w4a16_routed_expert_router_gb300 import _build, attention as at

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "moe_attn.h")


@pytest.fixture(scope="module")
def L():
    _build.build()
    return at._lib()


def test_header_declares_the_binding_names(L):
    names = set(re.findall(r"\b(moe_attn_[a-z0-9_]+)\s*\(", open(HEADER).read()))
    assert sorted(names) == sorted(moe.EXPORTS_ATTN)
    for name in names:
        assert hasattr(L, name), name


def test_binding_constants_match_the_header():
    text = open(HEADER).read()
    vals = {n: int(v, 0) for n, v in
            re.findall(r"#define\s+(MOE_ATTN_[A-Z0-9_]+)\s+(0x[0-9a-fA-F]+)u", text)}
    vals.update({n: int(v) for n, v in re.findall(r"\b(MOE_ATTN_[A-Z0-9_]+)\s*=\s*(-?\d+)", text)})
    assert len(vals) >= 14
    for name, v in vals.items():
        assert getattr(at, name, v) == v, name
        # statuses carry the values of the expert layer's
        other = name.replace("MOE_ATTN_", "MOE_W4A16_")
        if "ERR" in name and hasattr(moe, other):
            assert getattr(moe, other) == v


def test_structures_match_the_header(L):
    """Field names and their order, as declared."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name in ("rows", "rotation", "config", "cache", "batch", "scores"):
        body = re.search(r"typedef struct moe_attn_%s \{(.*?)\}" % name, text, re.S).group(1)
        fields = [f.strip(" *") for line in body.split(";") if line.strip()
                  for f in re.sub(r"^\s*(const\s+)?\w+\s*\**", "", line.strip()).split(",")]
        assert fields == [f for f, _ in getattr(at, "moe_attn_" + name)._fields_]


def _cfg(**kw):
    base = dict(q_heads=32, kv_heads=8, head_dim=128, page_size=16, max_tokens=64, max_seqs=8,
                dtype=0, flags=0)
    base.update(kw)
    return at.moe_attn_config(*[base[n] for n, _ in at.moe_attn_config._fields_])


@pytest.mark.parametrize("kw,status", [
    (dict(q_heads=0), -2), (dict(q_heads=33), -2), (dict(kv_heads=0), -2),
    (dict(q_heads=65, kv_heads=1), -2), (dict(head_dim=0), -2), (dict(head_dim=132), -2),
    (dict(head_dim=136), -2), (dict(page_size=8), -2), (dict(page_size=48), -2),
    (dict(page_size=512), -2), (dict(max_tokens=0), -1), (dict(max_tokens=(1 << 20) + 1), -1),
    (dict(max_seqs=0), -1), (dict(max_seqs=65537), -1), (dict(dtype=2), -1), (dict(flags=1), -1),
])
def test_invalid_configs_are_refused(L, kw, status):
    n, h = ctypes.c_size_t(), ctypes.c_void_p()
    assert L.moe_attn_workspace_bytes(_cfg(**kw), n) == status
    assert L.moe_attn_create(_cfg(**kw), 0, h) == status and not h.value


def test_workspace_and_null_arguments(L):
    n = ctypes.c_size_t()
    assert L.moe_attn_workspace_bytes(_cfg(), n) == 0 and n.value > 0
    assert L.moe_attn_workspace_bytes(None, n) == -1
    assert L.moe_attn_workspace_bytes(_cfg(), None) == -1
    assert L.moe_attn_create(_cfg(), 0, None) == -1
    assert L.moe_attn_destroy(None) == 0
    assert L.moe_attn_append(None, None, None, None, None, None, None, 0, None, None, None) == -1
    assert L.moe_attn_forward(None, None, None, None, None, None, None, None) == -1
    assert L.moe_attn_check_device_errors(None, None) == -1


def test_rope_refusals(L):
    r = at.moe_attn_rotation(8, 64, 0, 1.0, 0)
    row = at.moe_attn_rows(16, 128, 64)
    odd = at.moe_attn_rows(17, 128, 64)

    def call(x=row, out=row, pos=16, T=1, heads=2, dim=64, dtype=0, rot=r):
        return L.moe_attn_rope(x, out, pos, T, heads, dim, dtype, rot, None)

    assert call(T=0) == 0 and call(heads=0) == 0
    assert call(T=-1) == -1 and call(heads=-1) == -1 and call(dtype=2) == -1
    assert call(dim=0) == -2 and call(dim=257) == -2 and call(dim=62) == -2
    assert call(heads=65537) == -2
    assert call(rot=None) == -1 and call(x=None) == -1 and call(pos=None) == -1
    assert call(x=odd) == -4
    for bad in (at.moe_attn_rotation(8, 63, 0, 1.0, 0), at.moe_attn_rotation(8, -2, 0, 1.0, 0)):
        assert call(rot=bad) == -2
    for bad in (at.moe_attn_rotation(8, 64, 2, 1.0, 0), at.moe_attn_rotation(8, 64, 0, 1.0, 2),
                at.moe_attn_rotation(8, 64, 0, math.nan, 0),
                at.moe_attn_rotation(None, 64, 0, 1.0, 0)):
        assert call(rot=bad) == -1
    assert call(out=at.moe_attn_rows(20, 128, 64)) == -1  # overlaps x, shifted
    assert call(x=at.moe_attn_rows(16, -128, 64)) == -1


def test_frequencies():
    freq, mag = moe.moe_attn_rope_frequencies(128, device="cpu")
    assert mag == 1.0 and freq.shape == (64,)
    for i, f in enumerate(freq.tolist()):
        want = 10000.0 ** (-2 * i / 128) / (2 * math.pi) * 2.0 ** 64
        assert abs(f - want) <= 2.0 ** -50 * want + 1   # fp64 pow and division
    # interpolated positions: every pair slower by the factor
    lin, mag = moe.moe_attn_rope_frequencies(128, factor=4.0, device="cpu")
    assert mag == 1.0
    assert all(abs(4 * a - b) <= 2.0 ** -50 * b + 4 for a, b in zip(lin.tolist(), freq.tolist()))
    # by parts: fast pairs kept, slow ones divided, between them in between
    part, mag = moe.moe_attn_rope_frequencies(128, factor=8.0, by_parts=True, original_len=4096,
                                              device="cpu")
    assert abs(mag - (1 + 0.1 * math.log(8.0))) < 1e-6
    ratio = [a / b for a, b in zip(freq.tolist(), part.tolist())]
    turns = [4096 * f / 2.0 ** 64 for f in freq.tolist()]
    assert all(1 - 1e-12 <= a <= b + 1e-12 for a, b in zip(ratio, ratio[1:]))
    for t, x in zip(turns, ratio):
        assert x == pytest.approx(1.0 if t > 32 else 8.0 if t < 1 else x)
    assert moe.moe_attn_rope_frequencies(0, device="cpu")[0].shape == (0,)
    for kw in [dict(rot_dim=3), dict(rot_dim=258), dict(rot_dim=-2)]:
        with pytest.raises(moe.MoeError) as e:
            moe.moe_attn_rope_frequencies(device="cpu", **kw)
        assert e.value.status == -2
    for kw in [dict(base=1.0), dict(base=math.nan), dict(factor=0.5), dict(factor=math.inf),
               dict(by_parts=True, original_len=0.0),
               dict(by_parts=True, beta_fast=1.0, beta_slow=1.0)]:
        with pytest.raises(moe.MoeError) as e:
            moe.moe_attn_rope_frequencies(64, device="cpu", **kw)
        assert e.value.status == -1


def test_tensors_of_the_host_are_refused(L):
    import torch
    freq = moe.moe_attn_rope_frequencies(8, device="cpu")[0]
    x, pos = torch.zeros(2, 3, 8, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for args in [(x, pos, freq), (x.float(), pos, freq), (x[0], pos, freq)]:
        with pytest.raises(ValueError):
            moe.moe_attn_rope(*args)
    with pytest.raises(ValueError):
        moe.moe_attn_rope(x, pos, freq, layout="other")
    with pytest.raises(AttributeError):
        moe.moe_attn_rope(None, pos, freq)


def test_cache_bookkeeping():
    c = moe.PagedKvCache(5, 2, 16, 64, device="cpu")
    assert c.k_pages.shape == c.v_pages.shape == (5, 2, 16, 64)
    pos, slots = c.extend("a", 20)
    assert pos == list(range(20)) and len(set(slots)) == 20
    pos2, slots2 = c.extend("a", 13)
    assert pos2 == list(range(20, 33)) and not set(slots) & set(slots2)
    c.extend("b", 16)
    table, kv_len = c.tables(["b", "a", "none"])
    assert kv_len.tolist() == [16, 33, 0] and table.shape == (3, 3)
    for p, s in zip(pos + pos2, slots + slots2):
        assert s == int(table[1, p // 16]) * 16 + p % 16
    with pytest.raises(RuntimeError):
        c.extend("b", 17)
    assert c.length("b") == 16                      # a refused extension changes nothing
    with pytest.raises(RuntimeError):
        c.extend("new", 100)
    assert c.length("new") == 0 and c.tables(["new"])[1].tolist() == [0]
    with pytest.raises(ValueError):
        c.extend("a", -1)
    c.release("a")
    c.release("a")
    assert c.length("a") == 0 and len(c.extend("b", 64)[1]) == 64
    assert c.tables([])[0].shape[0] == 0


@pytest.mark.parametrize("device,index", [(None, 3), ("cuda", 3), ("cuda:0", 0), ("cuda:2", 2)])
def test_a_layer_without_a_device_number_is_on_the_current_one(L, monkeypatch, device, index):
    # as the cache's pages and the frequencies are
    import torch
    asked = []

    class Library:
        @staticmethod
        def moe_attn_create(cfg, device, out):
            asked.append(device)
            return at.MOE_ATTN_ERR_DEVICE

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(at, "_lib", lambda: Library)
    with pytest.raises(moe.MoeError):
        moe.PagedAttention(8, 2, 64, 16, 4, 4, device=device)
    assert asked == [index]
    with pytest.raises(ValueError):
        moe.PagedAttention(8, 2, 64, 16, 4, 4, device="cpu")


def test_layers_dropped_in_a_capture_are_destroyed_behind_it(L, monkeypatch):
    import gc
    import torch
    capturing, destroyed = [True], []

    class Library:
        @staticmethod
        def moe_attn_destroy(handle):
            assert not capturing[0]
            destroyed.append(handle.value)
            return 0

    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])

    def layer(address):
        a = object.__new__(moe.PagedAttention)
        a._library, a.handle = Library, ctypes.c_void_p(address)
        return a

    first, second = layer(8), layer(16)
    del first
    gc.collect()
    second.close()
    assert second.handle is None and destroyed == []
    second.close()
    capturing[0] = False
    layer(24).close()
    assert sorted(destroyed) == [8, 16, 24]
    second.close()
    assert len(destroyed) == 3


def test_a_stream_by_address_is_of_the_tensors_device(monkeypatch):
    import torch
    made, used = [], []

    class Tensor:
        def record_stream(self, stream):
            used.append(stream)

    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda address, device=None: made.append((address, device)) or "stream")
    device = torch.device("cuda", 1)
    at._in_use(4096, device, Tensor(), None, Tensor())
    assert made == [(4096, device)] and used == ["stream", "stream"]
