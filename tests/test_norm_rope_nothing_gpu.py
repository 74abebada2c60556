"""Gradients of norms and rotary positions where there are no tokens, or no heads: those
of the weights are zeros of the weights' shapes."""
import pytest
import torch

import w4a16_routed_expert_router_gb300 as moe
from tests import attn_cases as ac
from w4a16_routed_expert_router_gb300 import attention as at

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.lib()


@pytest.mark.parametrize("T,hq,hk", [(0, 2, 3), (5, 0, 2), (5, 2, 0), (5, 0, 0), (0, 0, 0)])
@pytest.mark.parametrize("stride", [0, 64])
def test_sums_over_nothing_are_written(T, hq, hk, stride):
    # by the C ABI, into memory that holds something else; what lies behind it stays
    L = at._lib()
    x = torch.randn(8, 4, 64, device=DEV).to(BF)
    dx = [torch.empty_like(x) for _ in range(2)]
    rows = [at.moe_attn_rows(t.data_ptr(), 4 * 64, 64) for t in (x, *dx)]
    freq, pos = ac.frequencies(64).to(DEV), torch.zeros(8, dtype=torch.int32, device=DEV)
    w = torch.ones(4, 64, device=DEV)
    norm = at.moe_attn_norm(w.data_ptr(), w.data_ptr(), stride, stride, 1e-6, 0.0, 1)
    r = at.moe_attn_rotation(freq.data_ptr(), 64, 0, 1.0, 0)
    dw = [torch.full((4, 64), 7.0, device=DEV) for _ in range(2)]
    n = at.ctypes.c_size_t()
    assert L.moe_attn_norm_rope_backward_bytes(T, hq, hk, 64, n) == 0
    work = torch.empty(n.value // 4 + 4, device=DEV)
    assert L.moe_attn_norm_rope_backward(
        rows[0], rows[0], rows[1], dw[0].data_ptr(), rows[0], rows[0], rows[2], dw[1].data_ptr(),
        pos.data_ptr(), T, hq, hk, 64, 0, norm, r, work.data_ptr(), n,
        torch.cuda.current_stream().cuda_stream) == 0
    for d, heads in zip(dw, (hq, hk)):
        used = heads if stride else 1
        assert bool((d[used:] == 7).all())
        if T == 0 or heads == 0:
            assert not d[:used].any()
        else:
            assert bool((d[:used] != 7).all())


@pytest.mark.parametrize("heads,shape", [(0, (64,)), (0, (0, 64)), (1, (64,)), (1, (1, 64))])
def test_gradients_have_the_weights_shapes(heads, shape):
    x, pos = torch.zeros(5, heads, 64, device=DEV, dtype=BF), torch.arange(5, device=DEV).int()
    k, freq = torch.randn(5, 2, 64, device=DEV).to(BF), ac.frequencies(64).to(DEV)
    w, wk = torch.ones(shape, device=DEV), torch.ones(64, device=DEV)
    held = [torch.full((64,), 7.0, device=DEV) for _ in range(8)]
    del held                                       # what new tensors may find
    dx, dk, dw, dwk = moe.moe_attn_norm_rope_backward(x, k, x, k, pos, freq, moe.HeadNorm(w, wk))
    assert dx.shape == x.shape and dw.shape == w.shape and dw.dtype == F32 and not dw.any()
    if not heads:
        alone = moe.moe_attn_norm_rope_backward(None, k, None, k, pos, freq,
                                                moe.HeadNorm(None, wk))
        assert torch.equal(alone[1], dk) and torch.equal(alone[3], dwk)
