"""The example decoder layer (examples/decoder_layer.py): the cache and the
attention compose with the routed-expert layer, and tokens that arrive in
chunks and one by one give what a whole prompt gives."""
import pytest
import torch

import moe_synth as ms

pytestmark = pytest.mark.gpu


def _layer(**kw):
    from examples.decoder_layer import DecoderLayer
    return DecoderLayer(ms.CONFIGS["tiny16"], 4, 2, 64, num_pages=64, max_tokens=512, **kw)


def test_chunks_and_single_tokens_give_the_whole_prompt():
    hidden = ms.CONFIGS["tiny16"].hidden
    x = torch.randn(150, hidden, device="cuda:0").to(torch.bfloat16)
    other = torch.randn(40, hidden, device="cuda:0").to(torch.bfloat16)
    layer = _layer()
    whole = layer.attention(x, ["w"], [150])
    parts = [layer.attention(torch.cat([x[:100], other[:30]]), ["p", "o"], [100, 30])[:100]]
    parts.append(layer.attention(torch.cat([other[30:], x[100:147]]), ["o", "p"], [10, 47])[10:])
    for t in range(147, 150):
        parts.append(layer.attention(x[t:t + 1], ["p"], [1]))
    got = torch.cat(parts).double()
    # the attention's results and the projection behind it are rounded to bf16
    # (2^-8 each) in both runs, from equal q, k, v and fp32 scores; the residual
    # sum is rounded once more: 2^-7 of the attention's part (below 4 in size)
    # and 2^-8 of the sum, twice
    bound = 4 * 2.0 ** -7 + 2 * 2.0 ** -8 * whole.double().abs()
    assert bool(((got - whole.double()).abs() <= bound).all())
    assert layer.check() == 0
    layer.cache.release("w")
    layer.close()


def test_forward_and_release():
    layer = _layer()
    hidden = ms.CONFIGS["tiny16"].hidden
    for counts in ([200, 1, 64], [1, 1, 1], [1, 30, 1]):
        y = layer.forward(torch.randn(sum(counts), hidden, device="cuda:0").to(torch.bfloat16),
                          ["a", "b", "c"], counts)
        assert y.shape == (sum(counts), hidden) and bool(torch.isfinite(y.float()).all())
    assert layer.check() == 0
    assert [layer.cache.length(s) for s in "abc"] == [202, 32, 66]
    layer.close()


def test_command_runs():
    from examples.decoder_layer import main
    assert main(["--steps", "2"]) == 0
