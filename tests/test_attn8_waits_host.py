"""In which order the tensor-core kernel over an 8-bit cache waits, checked in its
source. A wait goes by the parity of a barrier's phase, so it says something only where
the barrier is known to be in that phase or the one behind it. That holds for a tile's
products, which nobody else waits for; the scales' barriers are everybody's, and a tile
that passes pieces over may be several of their phases ahead: it waits for its products
of the block first, which are made from keys that come after all scales before them."""
import os
import re

from w4a16_routed_expert_router_gb300 import _build

SOURCE = re.sub(r"//[^\n]*", "", open(os.path.join(_build.CSRC, "attn8_tc.cu")).read())


def _role(first, last):
    return SOURCE[SOURCE.index(first):SOURCE.index(last)]


def test_products_are_waited_for_before_their_scales():
    softmax = SOURCE[SOURCE.index("kSoftmaxRegs8));"):]
    assert softmax.count("s.s_full") == softmax.count("s.sc_ready") == 1
    products, scales = softmax.index("s.s_full"), softmax.index("s.sc_ready")
    assert products < scales < softmax.index("s.scales[")


def test_scales_are_ready_before_the_next_keys():
    # what the order above relies on: a converting warp arrives for a block's keys, then
    # for its scales, and then goes on to the next block
    converter = _role("kConverterRegs));", "kOtherRegs8));")
    keys, scales = (converter.index(f"mbar_arrive(&s.{n}[") for n in ("kv_ready", "sc_ready"))
    assert converter.index("spread<ND>") < keys < scales
    blocks = converter.index("++block")
    assert blocks < keys and "sc_ready" not in converter[:blocks]
    # and products are issued from keys that are ready
    assert "bwait(&s.kv_ready[slot]" in SOURCE
