"""The example decoder layer in the norm: tokens in chunks and one by one against the
whole prompt, and the whole prompt against fp64.

Each rounding to bf16 moves a value by at most u = 2^-8 of itself, evenly spread:
u / sqrt(3) of the norm of independent values. A result of the layer's attention
half has on its way: the softmax's numerators, the attention's result and the
projection, each rounded once (of the attention's part a), and the residual sum s.
Products with weights are the library's, in fp32, whose order may differ from batch
to batch and so round q, k and v to a neighbour: counted as one more rounding each."""
import math

import pytest
import torch

import moe_synth as ms
from tests import attn_cases as ac

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


def _norms(layer, x, got, ref, runs):
    a = float((ref.double() - x.double()).norm())
    s = float(ref.double().norm())
    return float((got.double() - ref.double()).norm()), math.sqrt(
        runs / 3) * U * math.sqrt(6 * a * a + s * s), a


def _layer():
    from examples.decoder_layer import DecoderLayer
    return DecoderLayer(ms.CONFIGS["tiny16"], 4, 2, 64, num_pages=64, max_tokens=512)


def test_chunks_and_single_tokens_in_the_norm():
    layer = _layer()
    x = torch.randn(150, ms.CONFIGS["tiny16"].hidden, device="cuda:0").to(torch.bfloat16)
    whole = layer.attention(x, ["w"], [150])
    cuts = [0, 100, 147, 148, 149, 150]
    parts = torch.cat([layer.attention(x[a:b], ["p"], [b - a]) for a, b in zip(cuts, cuts[1:])])
    diff, bound, a = _norms(layer, x, parts, whole, runs=2)
    assert diff <= bound and bound < 0.1 * a    # the bound would see a tenth of it missing
    assert layer.check() == 0
    layer.close()


def test_whole_prompt_against_the_definition():
    from examples.decoder_layer import rms_norm
    layer = _layer()
    x = torch.randn(150, ms.CONFIGS["tiny16"].hidden, device="cuda:0").to(torch.bfloat16)
    got = layer.attention(x, ["w"], [150])
    qkv = (rms_norm(x).double() @ layer.w_qkv.double().T).view(150, -1, 64)
    pos = torch.arange(150)
    q, _ = ac.rotary(qkv[:, :4], pos, layer.freq.cpu(), "half")
    k, _ = ac.rotary(qkv[:, 4:6], pos, layer.freq.cpu(), "half")
    out, _, _ = ac.sequence(q, k, qkv[:, 6:].cpu(), 64 ** -0.5)
    want = x.double() + out.reshape(150, -1).to("cuda:0") @ layer.w_out.double().T
    diff, bound, a = _norms(layer, x, got, want, runs=1)
    assert diff <= bound and bound < 0.1 * a
    layer.close()
