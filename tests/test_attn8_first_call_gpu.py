"""A process whose first calls over an 8-bit cache are captured into graphs: their kernels
are loaded and set up then, which a capture must not mind."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch, w4a16_routed_expert_router_gb300 as moe
n = {n}
layer = moe.PagedAttention(8, 2, 128, 16, 4096, 2)
cache = moe.PagedKvCache(64, 2, 16, 128, dtype=torch.float8_e4m3fn)
freq = moe.moe_attn_rope_frequencies(128)[0]
q, k, v = (torch.randn(n, h, 128, device="cuda").bfloat16() for h in (8, 2, 2))
w = torch.ones(128, device="cuda")
pos, slots = cache.extend("s", n)
pos, slots = torch.tensor(pos, dtype=torch.int32).cuda(), torch.tensor(slots).cuda()
table, kv_len = cache.tables(["s"])
cu = torch.tensor([0, n], dtype=torch.int32).cuda()

def step():
    qn = layer.append(q, k, v, pos, slots, cache.k_pages, cache.v_pages, freq,
                      norm=moe.HeadNorm(w, w), **cache.scales)
    return layer.forward(qn, cache.k_pages, cache.v_pages, table, cu, kv_len, n, **cache.scales)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
torch.cuda.synchronize()
first = out.clone()
assert torch.isfinite(first).all() and first.any()
assert torch.equal(step(), first) and layer.check_device_errors() == 0
print("equal")
"""


@pytest.mark.parametrize("n", [3, 60, 700])     # few tokens, over codes, brought to 16 bits
def test_first_calls_are_captured(n):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", PROGRAM.format(n=n)], cwd=root, timeout=300,
                          capture_output=True, text=True)
    assert done.returncode == 0 and done.stdout.strip() == "equal", done.stderr[-2000:]
