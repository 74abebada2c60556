"""What the kernels of norms and of the 8-bit cache ask of a launch, without a GPU: their
launching functions linked against a runtime that records launches
(fake_launch_record.cu), and the kernels' own shared memory as the compiler tells it."""
import concurrent.futures as cf
import ctypes
import os
import random
import re
import subprocess

import pytest

from w4a16_routed_expert_router_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))
SHARED = 48 * 1024   # of a CTA, the kernel's own included, where no attribute says more


@pytest.fixture(scope="module")
def record(tmp_path_factory):
    """(library, {kernel: bytes of its own})."""
    out = tmp_path_factory.mktemp("record")
    files = [os.path.join(_build.CSRC, f) for f in ("norm_rope.cu", "cache8.cu")]
    files.append(os.path.join(HERE, "fake_launch_record.cu"))

    def compiled(src):
        obj = str(out / (os.path.basename(src) + ".o"))
        done = subprocess.run([_build.nvcc(), *_build.ARCH, *_build.FLAGS, "-Xptxas", "-v", "-I" +
                               _build.CSRC, "-c", src, "-o", obj], check=True, capture_output=True,
                              text=True)
        return obj, done.stderr + done.stdout

    with cf.ThreadPoolExecutor(3) as pool:
        objects, said = zip(*pool.map(compiled, files))
    # the rest of the runtime that compiled launches name: nothing calls it here, and
    # registering a variable does nothing
    rest = out / "rest.c"
    rest.write_text("".join(f"int __cuda{n}(void) {{ return 0; }}\n" for n in (
        "GetKernel", "LaunchKernel", "PopCallConfiguration", "RegisterVar")))
    lib = str(out / "record.so")
    subprocess.run(["gcc", "-O1", "-fPIC", "-c", str(rest), "-o", str(out / "rest.o")], check=True)
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", *objects, str(out / "rest.o"), "-o", lib],
                   check=True)
    own = {}
    for name, used in re.findall(r"entry function '(\w+)'.*?(Used [^\n]*)", "".join(said), re.S):
        m = re.search(r"(\d+) bytes smem", used)
        own[name] = int(m.group(1)) if m else 0
    L = ctypes.CDLL(lib)
    L.record_take.restype = ctypes.c_char_p
    return L, own


def shapes():
    rng = random.Random(5)
    dims = [(128, 128), (128, 64), (64, 64), (128, 32), (64, 32), (32, 32), (16, 16), (96, 24),
            (80, 80), (112, 20), (128, 0), (72, 8)]
    for tokens in (1, 63, 1216, 4863, 4864, 9728, 19456, 38912, 100003):   # where rules change
        for hq in (0, 1, 2, 3, 4, 5, 8, 32):
            for d, rot in dims:
                yield tokens, hq, rng.choice([1, 2, 8]), d, rot, rng.randint(0, 1)
    for _ in range(500):
        d = 8 * rng.randint(1, 16)
        yield (int(2 ** rng.uniform(0, 20)), rng.randint(0, 64), rng.randint(1, 16), d,
               2 * rng.randint(0, d // 2), rng.randint(0, 1))


@pytest.mark.parametrize("call", ["append8", "norm", "append_norm", "gradient"])
def test_no_launch_asks_for_more_than_there_is(record, call):
    L, own = record
    seen, most = set(), 0
    wide = [(t, hq, hk, 2 * d, 2 * r, il) for t, hq, hk, d, r, il in shapes()]
    for shape in list(shapes()) + (wide if call in ("norm", "gradient") else []):
        assert getattr(L, "record_" + call)(*shape) == 0
        for line in L.record_take().decode().split(";")[:-1]:
            name, *numbers = line.split()
            gx, gy, bx, by, bz, dynamic = map(int, numbers)
            assert own[name] + dynamic <= SHARED, (name, shape)
            assert 0 < gx < 2 ** 31 and 0 < gy < 65536 and 0 < bx * by * bz <= 1024 and bz <= 64
            seen.add(name)
            most = max(most, own[name] + dynamic)
    assert len(seen) >= 2
    if call != "gradient":
        assert most == SHARED    # the bound is met, not missed by far
