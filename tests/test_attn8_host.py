"""Host-side checks of include/moe_attn8.h: names, refusals before any device work,
the test definitions themselves. No kernel is launched here."""
import ctypes
import math
import os
import re

import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn8_cases as a8
from w4a16_routed_expert_router_gb300 import _build, attention as at

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "moe_attn8.h")


@pytest.fixture(scope="module")
def L():
    _build.build()
    return at._lib()


def test_header_declares_the_binding_names(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_attn_[a-z0-9_]+)\s*\(", text))
    assert sorted(names) == sorted(moe.EXPORTS_ATTN8)
    for name in names:
        assert hasattr(L, name), name
    assert sorted(at._signatures8()) == sorted(names)


def test_constants_and_structures_match_the_header(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert int(re.search(r"MOE_ATTN8_BLOCK (\d+)", text).group(1)) == at.MOE_ATTN8_BLOCK
    for n, v in re.findall(r"\b(MOE_ATTN_WEIGHT_\w+)\s*=\s*(\d+)", text):
        assert getattr(at, n) == int(v)
    for name in ("norm", "cache8", "extent"):
        body = re.search(r"typedef struct moe_attn_%s \{(.*?)\}" % name, text, re.S).group(1)
        fields = [f.strip(" *") for line in body.split(";") if line.strip()
                  for f in re.sub(r"^\s*(const\s+)?\w+\s*\**", "", line.strip()).split(",")]
        assert fields == [f for f, _ in getattr(at, "moe_attn_" + name)._fields_]


def _norm(**kw):
    base = dict(q_weight=64, k_weight=64, q_head_stride=0, k_head_stride=0, eps=1e-6, offset=0.0,
                weight_type=0)
    base.update(kw)
    return at.moe_attn_norm(*[base[n] for n, _ in at.moe_attn_norm._fields_])


BAD_NORMS = [(None, -1), (_norm(q_weight=None), -1), (_norm(k_weight=None), -1),
             (_norm(q_head_stride=-64), -1), (_norm(k_head_stride=63), -1),
             (_norm(eps=-1e-6), -1), (_norm(eps=math.inf), -1), (_norm(offset=math.nan), -1),
             (_norm(weight_type=2), -1), (_norm(q_weight=65), -4),
             (_norm(k_weight=66, weight_type=1), -4)]


def _rows(data, heads=2, dim=64):
    return at.moe_attn_rows(data, heads * dim, dim)


@pytest.mark.parametrize("norm,status", BAD_NORMS)
def test_bad_norms_are_refused(L, norm, status):
    r = at.moe_attn_rotation(8, 64, 0, 1.0, 0)
    x = _rows(1 << 20)
    assert L.moe_attn_norm_rope(x, x, x, x, 64, 0, 2, 2, 64, 0, norm, r, None) == status
    assert L.moe_attn_norm_rope_backward(x, x, x, 64, x, x, x, 64, 64, 1, 2, 2, 64, 0, norm, r,
                                         None, 0, None) == status


def test_norm_rope_refusals(L):
    r = at.moe_attn_rotation(8, 64, 0, 1.0, 0)
    q, k, qo, ko = (_rows(1 << n) for n in (20, 21, 22, 23))

    def call(q=q, qo=qo, k=k, ko=ko, pos=64, T=3, hq=2, hk=2, dim=64, dtype=0, norm=_norm(), rot=r):
        return L.moe_attn_norm_rope(q, qo, k, ko, pos, T, hq, hk, dim, dtype, norm, rot, None)

    assert call(T=0) == 0 and call(hq=0, hk=0) == 0 and call(q=None, qo=None, hk=0) == 0
    assert call(q=None, qo=None, k=None, ko=None) == 0
    assert call(T=-1) == -1 and call(hq=-1) == -1 and call(hk=-1) == -1 and call(dtype=2) == -1
    assert call(T=(1 << 30) + 1) == -3
    assert call(dim=0) == -2 and call(dim=257) == -2 and call(dim=62) == -2
    assert call(hq=65537) == -2 and call(hk=65537) == -2
    assert call(rot=None) == -1 and call(pos=None) == -1
    assert call(q=None) == -1 and call(qo=None) == -1 and call(k=None) == -1
    assert call(q=at.moe_attn_rows((1 << 20) + 1, 128, 64)) == -4
    assert call(qo=at.moe_attn_rows(1 << 22, 64, 64)) == -1        # rows on each other
    assert call(qo=at.moe_attn_rows((1 << 20) + 32, 128, 64)) == -1  # overlaps q, shifted
    # an output on the other input, or on the other output
    assert call(qo=_rows(1 << 21)) == -1 and call(ko=_rows(1 << 20)) == -1
    assert call(ko=_rows(1 << 22)) == -1
    # weights that no head needs are not looked at
    assert call(q=None, qo=None, T=0, norm=_norm(q_weight=None)) == 0


def test_slices_of_one_buffer_are_told_apart(L):
    """q, k and outputs inside the rows of one buffer, against the elements themselves."""
    import random
    rng = random.Random(3)
    r, n = at.moe_attn_rotation(64, 16, 0, 1.0, 0), _norm()
    seen = set()
    for _ in range(2000):
        T, hq, hk, step = rng.choice([1, 2, 3]), rng.choice([1, 2, 4]), rng.choice([1, 2]), 16 * 12
        at_q, at_k, at_qo, at_ko = (16 * rng.randint(0, 8) for _ in range(4))
        rows = [at.moe_attn_rows((1 << 20) + 2 * a, step, 16) for a in (at_q, at_k, at_qo, at_ko)]
        cells = [{a + t * step + h * 16 for t in range(T) for h in range(m)}
                 for a, m in ((at_q, hq), (at_k, hk), (at_qo, hq), (at_ko, hk))]
        q, k, qo, ko = cells
        bad = ((at_q != at_qo and q & qo) or (at_k != at_ko and k & ko) or qo & k or ko & q or
               qo & ko)
        # a workspace that is missing stands for a launch: it is refused last
        got = L.moe_attn_norm_rope_backward(rows[0], rows[0], rows[2], 64, rows[1], rows[1],
                                            rows[3], 64, 64, T, hq, hk, 16, 0, n, r, 8, 1 << 40,
                                            None)
        assert got == (-1 if bad else -4), (T, hq, hk, at_q, at_k, at_qo, at_ko)
        seen.add(bool(bad))
    assert len(seen) == 2


def test_gradient_refusals(L):
    r = at.moe_attn_rotation(8, 64, 0, 1.0, 0)
    n = ctypes.c_size_t()
    assert L.moe_attn_norm_rope_backward_bytes(7, 2, 2, 64, n) == 0 and n.value > 0
    assert L.moe_attn_norm_rope_backward_bytes(0, 2, 2, 64, n) == 0 and n.value == 0
    assert L.moe_attn_norm_rope_backward_bytes(7, 2, 2, 64, None) == -1
    assert L.moe_attn_norm_rope_backward_bytes(-1, 2, 2, 64, n) == -1
    assert L.moe_attn_norm_rope_backward_bytes(7, 2, 2, 300, n) == -2
    assert L.moe_attn_norm_rope_backward_bytes(1 << 30, 65536, 65536, 256, n) == 0
    assert n.value < 1 << 32                        # it follows the heads, not the tokens
    x, dx, y, dk = (_rows(1 << i) for i in (20, 21, 22, 23))

    def call(dq=y, q=x, dx=dx, dw=64, pos=64, ws=64, size=1 << 30):
        return L.moe_attn_norm_rope_backward(dq, q, dx, dw, None, None, None, None, pos, 7, 2, 2,
                                             64, 0, _norm(), r, ws, size, None)

    assert call(dq=None) == -1 and call(q=None) == -1 and call(dx=None) == -1 and call(dw=None) == -1
    assert call(pos=None) == -1 and call(ws=None) == -1 and call(size=15) == -1
    assert call(dw=66) == -4 and call(ws=72) == -4
    assert call(dx=at.moe_attn_rows((1 << 22) + 32, 128, 64)) == -1


def test_null_handles_are_refused(L):
    assert L.moe_attn_append_norm(*[None] * 7, 0, None, None, None, None) == -1
    assert L.moe_attn_append8(*[None] * 7, 0, None, None, None, None) == -1
    assert L.moe_attn_read8(*[None] * 6) == -1
    assert L.moe_attn_forward8(*[None] * 7, 0, None, 0, None) == -1
    assert L.moe_attn_forward8_scratch_bytes(None, None, None) == -1
    assert L.moe_attn_forward_sinks(*[None] * 7, 0, None) == -1


def test_python_refusals(L):
    freq = moe.moe_attn_rope_frequencies(8, device="cpu")[0]
    x, pos = torch.zeros(2, 3, 8, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    w = torch.ones(8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_attn_norm_rope(x, None, pos, freq, moe.HeadNorm(w, w))       # of the host
    with pytest.raises(ValueError, match="HeadNorm"):
        moe.moe_attn_norm_rope(x, None, pos, freq, (w, w, 1e-6, 0.0))
    with pytest.raises(ValueError, match="HeadNorm"):
        moe.moe_attn_norm_rope_backward(x, None, x, None, pos, freq, None)
    with pytest.raises(ValueError, match="torch stream"):
        moe.moe_attn_norm_rope_backward(x, None, x, None, pos, freq, moe.HeadNorm(w, w), stream=64)
    with pytest.raises(ValueError, match="needed"):
        moe.moe_attn_norm_rope(None, None, pos, freq, moe.HeadNorm(w, w))
    with pytest.raises(ValueError, match="needed"):
        moe.moe_attn_norm_rope_backward(None, None, None, None, pos, freq, moe.HeadNorm(w, w))


def test_cache_of_8_bits():
    c = moe.PagedKvCache(5, 2, 32, 64, dtype=torch.float8_e4m3fn, device="cpu")
    assert c.k_pages.dtype == torch.float8_e4m3fn
    assert sorted(c.scales) == ["k_scales", "v_scales"]
    for s in c.scales.values():
        assert s.shape == (5, 2, 2) and s.dtype == torch.float32 and not s.any()
    assert moe.PagedKvCache(5, 2, 32, 64, device="cpu").scales == {}


def test_the_definition_of_the_codes():
    """The tests' own rounding against torch's conversion, ties and edges included."""
    every = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(a8.F8).float()
    finite = every[every.isfinite()].double()
    assert torch.equal(a8.nearest(finite), finite)
    x = torch.cat([finite, (a8.VALUE[1:] + a8.VALUE[:-1]) / 2, torch.randn(4000).double() * 100,
                   torch.randn(4000).double() / 100]).clamp(-448, 448)
    assert torch.equal(a8.nearest(x), x.float().to(a8.F8).float().double())
    for top, want in ((448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (0.0, 2.0 ** -64),
                      (1e30, 2.0 ** 64), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8), (1.76, 2.0 ** -7)):
        assert float(a8.scale_for(torch.tensor([top]))[0]) == want
