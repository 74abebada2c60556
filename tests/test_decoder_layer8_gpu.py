"""The example decoder layer with norms of its heads, an 8-bit cache, a window and first
tokens that stay visible: tokens that arrive in chunks and one by one give what a whole
prompt gives, up to what 8 bits hold."""
import pytest
import torch

import moe_synth as ms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(norm=True, window=40, sinks=3),
                                dict(norm=True, cache8=True),
                                dict(cache8=True, window=40, sinks=3)])
def test_chunks_and_single_tokens_give_the_whole_prompt(kw):
    from examples.decoder_layer import DecoderLayer
    shape = ms.CONFIGS["tiny16"]
    layer = DecoderLayer(shape, 4, 2, 64, num_pages=64, max_tokens=512, **kw)
    x = torch.randn(150, shape.hidden, device="cuda:0").to(torch.bfloat16)
    whole = layer.attention(x, ["w"], [150]).double()
    parts = [layer.attention(x[:100], ["p"], [100]), layer.attention(x[100:147], ["p"], [47])]
    parts += [layer.attention(x[t:t + 1], ["p"], [1]) for t in range(147, 150)]
    got = torch.cat(parts).double()
    # bf16 as in the 16-bit cache's test: each run's attention and projection round to
    # bf16, 2^-7 of the attention's part (below 4 in size) and 2^-8 of the sum, twice.
    # Codes are the same in both runs but where a block's scale grows after some of its
    # rows were written, or seen: then those that are subnormal by the larger scale differ
    # by a step, 2^-9 of it, where the block's largest value is 224 of it or more. Values
    # are below 8, so that is below 8e-5 of each, 64 of them and a scale of 1 / 8 in a
    # score: small beside the roundings above.
    bound = 4 * 2.0 ** -7 + 2 * 2.0 ** -8 * whole.abs()
    assert bool(((got - whole).abs() <= bound).all())
    assert layer.check() == 0
    layer.close()


def test_command_runs():
    from examples.decoder_layer import main
    assert main(["--steps", "2", "--norm", "--cache8", "--window", "64", "--sinks", "4"]) == 0
