"""How the tensor-core attention kernel ends after a wait that gave up, checked in
its source: the warps of a softmax group meet at named barriers, which wait
without a limit, so no warp may leave its pieces, or pass into the code with
those barriers, on the outcome of a wait of its own."""
import os
import re

from w4a16_routed_expert_router_gb300 import _build

SOURCE = open(os.path.join(_build.CSRC, "attn_tc.cu")).read()


def _plain(text):
    return re.sub(r"//[^\n]*", "", text)


def _block(text, at):
    """(start, end) of the braces that open first at or behind `at`."""
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return start, i
    raise AssertionError("unbalanced braces")


def _softmax_role():
    at = SOURCE.index("// ---------------------------------------------------------------- softmax")
    text = _plain(SOURCE[at:])
    return text[:text.index("__syncthreads()")]


def _piece_loop():
    role = _softmax_role()
    heads = [m for m in re.finditer(r"\b(for|while)\s*\(", role)]
    start, end = _block(role, heads[0].end())
    assert "finish_piece" in role[start:end]
    return role[heads[0].start():start], role[start + 1:end]


def test_a_group_leaves_its_pieces_as_one():
    head, body = _piece_loop()
    assert "hold" not in head and "wait" not in head
    inner = []
    for m in re.finditer(r"\b(for|while)\s*\([^{;]*;?[^{;]*;?[^{;]*\)\s*\{", body):
        inner.append(_block(body, m.start()))
    exits = [m.start() for m in re.finditer(r"\b(break|return|goto)\b", body)
             if not any(a < m.start() < b for a, b in inner)]
    # the first vote of a piece is every warp's, and so is one where a warp leaves
    assert re.match(r"\s*const Piece\* held = pieces\.hold\(\);\s*if \(!group_all", body)
    assert [re.search(r"if \(([^{};]*)\)\s*$", body[:at]).group(1) for at in exits] == [
        "!group_all(t, held != nullptr)", "(!ok || held->pieces) && !group_all(t, ok)"]


def test_named_barriers_are_met_by_the_whole_group():
    _, body = _piece_loop()
    call = body.index("finish_piece")
    # no warp comes here but after a vote where there are barriers (split items)
    assert re.search(r"if \(\(!ok \|\| held->pieces\) && !group_all\(t, ok\)\) break;\s*$",
                     body[:call])
    at = SOURCE.index("void finish_piece(")
    start, end = _block(SOURCE, at)
    finish = _plain(SOURCE[start:end])
    assert finish.index("if (g.pieces)") < finish.index("bar.sync") < finish.index("if (holds)")
    assert "group_sync" not in finish[finish.index("if (holds)"):]
    # nothing in there gives up: no bounded wait, no way out
    assert not re.search(r"\b(bwait|bwait_piece|warp_wait|mbar_wait|goto)\b|\breturn\s*;", finish)
    # and the only other named barrier of the kernel is the vote itself
    assert len(re.findall(r"\bbar(?:rier)?\.(?:cta\.)?(?:sync|red|arrive)", _plain(SOURCE))) == 2


def test_waits_are_bounded():
    # every wait on an mbarrier goes by the helpers with a limit
    assert not re.search(r"\bmbar_try_wait|mbarrier\.(test|try)_wait", _plain(SOURCE))
