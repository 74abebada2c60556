"""The host side of the attention operators' C ABI (csrc/attn.cu) against a
stand-in for the CUDA runtime (fake_cudart.cpp): what it asks of the runtime, in
which order, on which device, and what it makes of errors. No GPU takes part."""
import ctypes
import os
import subprocess

import pytest

from w4a16_routed_expert_router_gb300 import _build, attention as at

HERE = os.path.dirname(os.path.abspath(__file__))
TIMEOUT, RANGE = at.MOE_ATTN_DEVERR_TIMEOUT, at.MOE_ATTN_DEVERR_RANGE


@pytest.fixture(scope="module")
def F(tmp_path_factory):
    out = tmp_path_factory.mktemp("fake")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc())))
    runtime = os.path.join(HERE, "fake_cudart.cpp")
    jobs = [["g++", "-std=c++17", "-O1", "-fPIC", "-I" + os.path.join(cuda, "include"), "-c",
             runtime]]
    for src in (os.path.join(_build.CSRC, "attn.cu"), os.path.join(HERE, "fake_launches.cu")):
        jobs.append([_build.nvcc(), *_build.ARCH, *_build.FLAGS, "-I" + _build.CSRC, "-c", src])
    objects = [str(out / f"{i}.o") for i in range(len(jobs))]
    for job, obj in zip(jobs, objects):
        subprocess.run([*job, "-o", obj], check=True)
    lib = str(out / "fake.so")
    # its own calls go to its own functions, whatever else the process has loaded
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", *objects, "-o", lib], check=True)
    L = ctypes.CDLL(lib)
    at.register(L)
    L.fake_calls.restype = ctypes.c_char_p
    L.fake_counters.restype = ctypes.c_void_p
    L.fake_fail.argtypes = [ctypes.c_char_p]
    return L


class Handle:
    """A handle on device 1 while device 0 is current; calls by ctypes."""

    def __init__(self, F, device=1):
        self.F = F
        F.fake_reset()
        F.fake_use(0)
        self.cfg = at.moe_attn_config(8, 2, 64, 16, 64, 8, 0, 0)
        self.h = ctypes.c_void_p()
        assert F.moe_attn_create(self.cfg, device, self.h) == 0
        ws = ctypes.c_void_p.from_address(self.h.value + ctypes.sizeof(self.cfg) + 8).value
        n = ctypes.c_size_t()
        assert F.moe_attn_workspace_bytes(self.cfg, n) == 0
        self.words = (ctypes.c_uint32 * (n.value // 4)).from_address(ws)
        self.created = self.calls()

    def calls(self):
        got = self.F.fake_calls().decode().split(";")[:-1]
        self.F.fake_reset()
        return got

    def forward(self, max_q):
        rows = lambda a: at.moe_attn_rows(a, 8 * 64, 64)  # noqa: E731
        cache = at.moe_attn_cache(1 << 20, 1 << 21, 9, 2 * 16 * 64, 64, 16 * 64)
        batch = at.moe_attn_batch(64, 64, 64, 4, 4, 1, max_q, max_q)
        return self.F.moe_attn_forward(self.h, rows(1 << 22), rows(1 << 23), None, cache, batch,
                                       at.moe_attn_scores(0.125, 0.0, 0, None, None), None)

    def append(self):
        rows = lambda a: at.moe_attn_rows(a, 2 * 64, 64)  # noqa: E731
        cache = at.moe_attn_cache(1 << 20, 1 << 21, 9, 2 * 16 * 64, 64, 16 * 64)
        return self.F.moe_attn_append(self.h, None, None, rows(1 << 22), rows(1 << 23), 64, 64, 1,
                                      at.moe_attn_rotation(64, 64, 0, 1.0, 0), cache, None)

    def check(self):
        flags = ctypes.c_uint32()
        return self.F.moe_attn_check_device_errors(self.h, flags), flags.value

    def counters(self, kernel):
        return (ctypes.c_uint32 * self.F.fake_counter_words(kernel)).from_address(
            self.F.fake_counters(kernel))


def test_a_new_handle_counts_from_zero(F):
    h = Handle(F)
    assert not any(h.words[:4096])
    assert h.forward(1) == 0 and h.forward(40) == 0
    for kernel in (0, 1):
        assert not any(h.counters(kernel))
    assert F.moe_attn_destroy(h.h) == 0


@pytest.mark.parametrize("bits", [TIMEOUT, TIMEOUT | RANGE])
def test_after_a_timeout_joins_count_from_zero(F, bits):
    # a launch that winds down leaves counters raised that only the second half of
    # a pair resets
    h = Handle(F)
    assert h.forward(1) == 0 and h.forward(40) == 0
    for kernel in (0, 1):
        c = h.counters(kernel)
        for i in range(len(c)):
            c[i] = 1 + i % 2
    h.words[0] = bits
    assert h.check() == (-6, bits)
    for kernel in (0, 1):
        assert not any(h.counters(kernel))
    assert h.check() == (0, 0)
    assert F.moe_attn_destroy(h.h) == 0


def test_without_a_timeout_counters_are_left_alone(F):
    h = Handle(F)
    assert h.forward(40) == 0
    h.counters(1)[3] = 1  # a launch that is under way elsewhere would own it
    h.words[0] = RANGE
    assert h.check() == (-6, RANGE) and h.counters(1)[3] == 1
    assert F.moe_attn_destroy(h.h) == 0


def test_cleared_memory_is_waited_for(F):
    # a memset returns before it has run, and streams other than the legacy one do
    # not wait for it: create and check return behind a synchronisation
    h = Handle(F)
    assert h.created[-2:] == ["memset", "sync"]
    for bits in (RANGE, TIMEOUT):
        h.words[0] = bits
        assert h.check()[1] == bits
        calls = h.calls()
        assert calls[0] == "sync" and calls[-2:] == ["memset", "sync"]
    h.check()
    assert h.calls() == ["sync", "memcpy"]
    assert F.moe_attn_destroy(h.h) == 0


@pytest.mark.parametrize("what", ["decode setup", "tc setup", "malloc", "memset", "sync"])
def test_create_reports_a_failing_call(F, what):
    F.fake_reset()
    F.fake_fail(what.encode())
    h = ctypes.c_void_p()
    assert F.moe_attn_create(at.moe_attn_config(8, 2, 64, 16, 64, 8, 0, 0), 0, h) == -5
    assert not h.value
    F.fake_reset()


def test_calls_run_on_the_handles_device_and_leave_the_callers(F):
    h = Handle(F, device=1)                 # device 0 is current throughout
    assert F.fake_device() == 0
    for call, launch in ((lambda: h.forward(1), "decode on 1"), (lambda: h.forward(40), "tc on 1"),
                         (h.append, "rope on 1")):
        assert call() == 0 and h.calls() == [launch]
        assert F.fake_device() == 0
        F.fake_fail(launch.split()[0].encode())  # a launch that fails
        assert call() == -5
        assert F.fake_device() == 0
        F.fake_reset()
    assert h.check() == (0, 0) and F.fake_device() == 0
    assert F.moe_attn_destroy(h.h) == 0 and F.fake_device() == 0
    F.fake_fail(b"malloc")
    out = ctypes.c_void_p()
    assert F.moe_attn_create(h.cfg, 1, out) == -5 and F.fake_device() == 0
    F.fake_reset()


@pytest.mark.parametrize("token,head,status", [
    (512, 64, 0), (64, 128, 0), (1000, 72, 0), (64, 512, 0), (100, 200, 0), (0, 64, -1),
    (128, 0, -1), (32, 256, -1), (256, 56, -1), (128, 64, -1), (450, 72, -1), (250, 72, -1),
    (504, 72, -1), (570, 72, 0)])
def test_outputs_whose_rows_lie_on_each_other_are_refused(F, token, head, status):
    at_rows = [set(range(t * token + h * head, t * token + h * head + 64))
               for t in range(2) for h in range(8)]
    assert (status == 0) == (len(set.union(*at_rows)) == 2 * 8 * 64)
    # q and out apart, 8 heads of 64; a turn in place of such rows as well
    h = Handle(F)
    x, out = at.moe_attn_rows(1 << 22, 512, 64), at.moe_attn_rows(1 << 23, token, head)
    r = at.moe_attn_rotation(64, 64, 0, 1.0, 0)
    assert F.moe_attn_rope(x, out, 64, 2, 8, 64, 0, r, None) == status
    assert F.moe_attn_rope(out, out, 64, 2, 8, 64, 0, r, None) == status
    # one row of each is no matter
    assert F.moe_attn_rope(x, at.moe_attn_rows(1 << 23, 0, 0), 64, 1, 1, 64, 0, r, None) == 0
    kv = at.moe_attn_rows(1 << 24, 128, 64)
    cache = at.moe_attn_cache(1 << 20, 1 << 21, 9, 2 * 16 * 64, 64, 16 * 64)
    assert F.moe_attn_append(h.h, x, out, kv, kv, 64, 64, 2, r, cache, None) == status
    batch = at.moe_attn_batch(64, 64, 64, 4, 4, 1, 2, 2)
    if token % 8 == 0 and head % 8 == 0:
        assert F.moe_attn_forward(h.h, x, out, None, cache, batch,
                                  at.moe_attn_scores(0.125, 0.0, 0, None, None), None) == status
    assert F.moe_attn_destroy(h.h) == 0


def test_long_outputs_are_checked_in_no_time(F):
    # a million tokens in between the heads, and heads in between the tokens
    r = at.moe_attn_rotation(64, 64, 0, 1.0, 0)
    for token, head, n, heads in ((64, 64 << 20, 1 << 20, 8), (64 * 8, 64, 1 << 20, 8),
                                  (64, 0, 1 << 20, 1), (0, 64, 1, 65536)):
        x, out = at.moe_attn_rows(0, token, head), at.moe_attn_rows(1 << 40, token, head)
        x.data = 1 << 22
        assert F.moe_attn_rope(x, out, 64, n, heads, 64, 0, r, None) == 0


def test_single_tokens_run_where_the_tensor_core_kernel_does_not(F):
    # built with other registers than its warps hand each other, it would wait for
    # ever: it is refused, and only it
    F.fake_reset()
    F.fake_fail(b"tc usable")
    h = ctypes.c_void_p()
    assert F.moe_attn_create(at.moe_attn_config(8, 2, 64, 16, 64, 8, 0, 0), 0, h) == 0
    F.fake_reset()
    handle = object.__new__(Handle)
    handle.F, handle.h = F, h
    assert handle.forward(1) == 0 and handle.calls() == ["decode on 0"]
    assert handle.append() == 0 and handle.calls() == ["rope on 0"]
    assert handle.forward(40) == -5 and handle.calls() == []
    assert F.moe_attn_destroy(h) == 0


def test_parts_of_one_buffer_do_not_overlap(F):
    # inputs and outputs with the same strides: against the elements themselves
    import random
    rng = random.Random(4)
    r = at.moe_attn_rotation(16, 16, 0, 1.0, 0)
    seen = set()
    for _ in range(3000):
        T, H = rng.choice([1, 2, 3, 5]), rng.choice([1, 2, 4])
        a, b = 16 + rng.choice([0, 0, 8, 16, 100]), rng.choice([1, 2, 3]) * 24
        token, head = (H * a + b, a) if rng.random() < 0.6 else (a, T * a + b)
        off = rng.choice([rng.randint(-200, 200), 16 * rng.randint(-12, 12), b, a, token, head])
        x, out = at.moe_attn_rows(1 << 20, token, head), at.moe_attn_rows((1 << 20) + 2 * off,
                                                                          token, head)
        rows = [t * token + h * head for t in range(T) for h in range(H)]
        if off == 0:
            want = 0                      # in place
        else:
            want = -1 if any(abs(off + p - q) < 16 for p in rows for q in rows) else 0
        assert F.moe_attn_rope(x, out, 64, T, H, 16, 0, r, None) == want, (T, H, token, head, off)
        seen.add((want, off == 0))
    assert len(seen) == 3
    # the queries and the results of one buffer, a slice each
    h = Handle(F)
    cache = at.moe_attn_cache(1 << 20, 1 << 21, 9, 2 * 16 * 64, 64, 16 * 64)
    batch = at.moe_attn_batch(64, 64, 64, 4, 4, 1, 40, 40)
    q, o = at.moe_attn_rows(1 << 22, 20 * 64, 64), at.moe_attn_rows((1 << 22) + 8 * 128, 20 * 64, 64)
    scores = at.moe_attn_scores(0.125, 0.0, 0, None, None)
    assert F.moe_attn_forward(h.h, q, o, None, cache, batch, scores, None) == 0
    o.data -= 128
    assert F.moe_attn_forward(h.h, q, o, None, cache, batch, scores, None) == -1
    assert F.moe_attn_destroy(h.h) == 0
