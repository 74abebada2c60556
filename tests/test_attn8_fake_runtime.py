"""The host side of include/moe_attn8.h (csrc/attn8.cu) against a stand-in for the CUDA
runtime (fake_cudart.cpp, fake_launches.cu, fake_launches8.cu): what is refused, and what
is launched. No GPU takes part."""
import concurrent.futures as cf
import ctypes
import os
import random
import subprocess

import pytest

from w4a16_routed_expert_router_gb300 import _build, attention as at

HERE = os.path.dirname(os.path.abspath(__file__))
HEADS, DIM, PAGE = 2, 64, 64


@pytest.fixture(scope="module")
def F(tmp_path_factory):
    out = tmp_path_factory.mktemp("fake8")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc())))
    jobs = [["g++", "-std=c++17", "-O1", "-fPIC", "-I" + os.path.join(cuda, "include"), "-c",
             os.path.join(HERE, "fake_cudart.cpp")]]
    for src in (os.path.join(_build.CSRC, "attn.cu"), os.path.join(_build.CSRC, "attn8.cu"),
                os.path.join(HERE, "fake_launches.cu"), os.path.join(HERE, "fake_launches8.cu")):
        jobs.append([_build.nvcc(), *_build.ARCH, *_build.FLAGS, "-I" + _build.CSRC, "-c", src])
    objects = [str(out / f"{i}.o") for i in range(len(jobs))]
    with cf.ThreadPoolExecutor(len(jobs)) as pool:
        list(pool.map(lambda j: subprocess.run([*j[0], "-o", j[1]], check=True),
                      zip(jobs, objects)))
    lib = str(out / "fake8.so")
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", *objects, "-o", lib], check=True)
    L = ctypes.CDLL(lib)
    at.register(L)
    at.register8(L)
    L.fake_calls.restype = ctypes.c_char_p
    L.fake_fail.argtypes = [ctypes.c_char_p]
    return L


class Handle:
    """A handle on device 1 while device 0 is current."""

    def __init__(self, F):
        self.F = F
        F.fake_reset()
        F.fake_use(0)
        self.h = ctypes.c_void_p()
        cfg = at.moe_attn_config(8, HEADS, DIM, PAGE, 4096, 8, 0, 0)
        assert F.moe_attn_create(cfg, 1, self.h) == 0
        self.calls()

    def calls(self):
        got = self.F.fake_calls().decode().split(";")[:-1]
        self.F.fake_reset()
        return got

    def cache(self, pages=9, codes=(HEADS * PAGE * DIM, DIM, PAGE * DIM), scales=(8, 4, 1)):
        """codes: strides of pages, tokens, heads; scales: of pages, heads, blocks"""
        return at.moe_attn_cache8(1 << 30, 1 << 32, 1 << 20, 1 << 21, pages, *codes, *scales)

    def append(self, cache):
        rows = lambda a: at.moe_attn_rows(a, HEADS * DIM, DIM)  # noqa: E731
        return self.F.moe_attn_append8(self.h, None, None, rows(1 << 22), rows(1 << 23), 64, 64, 1,
                                       None, at.moe_attn_rotation(64, 64, 0, 1.0, 0), cache, None)

    def read(self, cache):
        rows = lambda a: at.moe_attn_rows(a, HEADS * DIM, DIM)  # noqa: E731
        return self.F.moe_attn_read8(self.h, cache, at.moe_attn_extent(64, 64, 64, 4, 4, 1, 5),
                                     rows(1 << 22), rows(1 << 23), None)

    def forward(self, max_q, cache=None):
        rows = lambda a: at.moe_attn_rows(a, 8 * DIM, DIM)  # noqa: E731
        batch = at.moe_attn_batch(64, 64, 64, 4, 4, 1, max_q, max_q)
        return self.F.moe_attn_forward8(self.h, rows(1 << 22), rows(1 << 23), None,
                                        cache or self.cache(), batch,
                                        at.moe_attn_scores(0.125, 0.0, 0, None, None), 0, None, 0,
                                        None)


def test_a_cache_that_lies_on_itself_is_not_appended_to(F):
    # against the places themselves: of scales, and of codes in units of 16 bytes
    h, rng, seen = Handle(F), random.Random(6), set()
    for _ in range(4000):
        pages = rng.choice([1, 2, 3])
        s = rng.choice([(8, 4, 1), (4, 4 * pages, 1), (1, pages * 4, pages), (16, 8, 2), (0, 4, 1),
                        (8, 0, 1), (8, 4, 0), tuple(rng.randint(0, 20) for _ in range(3))])
        c = rng.choice([(HEADS * PAGE * DIM, DIM, PAGE * DIM), (HEADS * PAGE * DIM, HEADS * DIM, DIM),
                        (4 * PAGE * DIM, DIM, PAGE * DIM), (PAGE * DIM, DIM, PAGE * DIM),
                        (HEADS * PAGE * DIM, DIM, DIM), (HEADS * PAGE * DIM, 48, PAGE * DIM),
                        (HEADS * PAGE * DIM + 16, DIM, PAGE * DIM)])
        cache = h.cache(pages, c, s)
        scales = [p * s[0] + a * s[1] + b * s[2] for p in range(pages) for a in range(HEADS)
                  for b in range(PAGE // 16)]
        codes = [p * c[0] + t * c[1] + a * c[2] + i for p in range(pages) for a in range(HEADS)
                 for t in range(PAGE) for i in range(0, DIM, 16)]
        apart = len(set(scales)) == len(scales) and len(set(codes)) == len(codes)
        got = h.append(cache)
        if got == 0:
            assert apart, (pages, c, s)
        elif apart:      # refused all the same: places that go in between each other
            order = sorted(n for n, m in zip(s, (pages, HEADS, PAGE // 16)) if m > 1)
            assert got == -1 and order != sorted((8, 4, 1)) and s not in ((16, 8, 2),)
        assert got in (0, -1) and h.read(cache) == 0     # reading is nobody's harm
        seen.add((apart, got))
    assert {(True, 0), (False, -1)} <= seen and (False, 0) not in seen
    # usual layouts
    for s in ((8, 4, 1), (4, 4 * 9, 1), (1, 4 * 9, 9), (16, 8, 2), (2050, 4, 1)):
        assert h.append(h.cache(9, scales=s)) == 0, s
    for c in ((HEADS * PAGE * DIM, DIM, PAGE * DIM), (HEADS * PAGE * DIM, HEADS * DIM, DIM),
              (2 * HEADS * PAGE * DIM, 2 * DIM, 2 * PAGE * DIM)):
        assert h.append(h.cache(9, codes=c)) == 0, c
    assert F.moe_attn_destroy(h.h) == 0


def test_keys_and_values_in_one_place_are_not_appended(F):
    h = Handle(F)
    for twin in (("k", "v"), ("k_scales", "v_scales")):
        cache = h.cache()
        setattr(cache, twin[1], getattr(cache, twin[0]))
        assert h.append(cache) == -1 and h.read(cache) == 0
    assert h.append(h.cache()) == 0
    assert F.moe_attn_destroy(h.h) == 0


def test_kernels_are_set_up_once_for_a_handle(F):
    h = Handle(F)
    setup = ["decode8 setup", "tc8 usable", "tc8 setup"]
    assert h.forward(1) == 0 and h.calls() == setup + ["decode8 on 1"]
    assert h.forward(40) == 0 and h.forward(1) == 0 and h.calls() == ["tc8 on 1", "decode8 on 1"]
    assert F.moe_attn_destroy(h.h) == 0


@pytest.mark.parametrize("what", ["decode8 setup", "tc8 setup"])
def test_a_set_up_that_failed_is_made_again(F, what):
    h = Handle(F)
    F.fake_fail(what.encode())
    assert h.forward(1) == -5 and "decode8 on 1" not in h.calls()
    assert h.forward(1) == 0 and h.calls()[-1] == "decode8 on 1"
    assert F.moe_attn_destroy(h.h) == 0


def test_single_tokens_run_where_the_tensor_core_kernel_does_not(F):
    h = Handle(F)
    F.fake_fail(b"tc8 usable")
    assert h.forward(1) == 0 and h.calls()[-1] == "decode8 on 1"
    assert h.forward(40) == -5 and h.calls() == [] and h.forward(1) == 0
    assert F.moe_attn_destroy(h.h) == 0
