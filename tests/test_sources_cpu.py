"""Orderings that no run can show reliably, read from the kernels' sources."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_tensor_core_persistent_gb300", "csrc")


def functions(path):
    """(name, body) of the device functions of a source, comments taken out."""
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"__forceinline__\s+[\w:&*<> ]+?\b(\w+)\s*\([^{};]*\)\s*(?:const\s*)?\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), text[m.end():i - 1]


def test_lanes_that_asked_different_barriers_meet_at_a_warp_barrier():
    """Where the lanes of a warp wait on different mbarriers, a vote does not
    order memory between them: a __syncwarp has to stand between the last vote
    and every way out."""
    seen = 0
    for name in sorted(os.listdir(CSRC)):
        for fn, body in functions(os.path.join(CSRC, name)):
            if "try_wait(" not in body or "__all_sync(" not in body or not re.search(r"\?\s*bar\d", body):
                continue
            seen += 1
            last_vote = body.rindex("__all_sync(")
            barrier = body.find("__syncwarp()", last_vote)
            assert barrier > 0, f"{name}: {fn} leaves after a vote"
            assert "return" not in body[:barrier], f"{name}: {fn} leaves before the warp barrier"
    assert seen >= 1


def test_a_warp_barrier_follows_every_wait_of_half_a_warp():
    """On the way from each such wait to the caller, taken or not, stands a
    __syncwarp: after the first try, and after the long wait."""
    seen = 0
    for name in sorted(os.listdir(CSRC)):
        for fn, body in functions(os.path.join(CSRC, name)):
            if "try_wait(" not in body or "__all_sync(" not in body or not re.search(r"\?\s*bar\d", body):
                continue
            seen += 1
            for wait in re.finditer(r"\b(?:mbar_try_wait|spin)\(", body):
                after = body[wait.end():]
                barrier = after.find("__syncwarp()")
                assert barrier >= 0, f"{name}: {fn}"
                between = after[:barrier]
                assert "return" not in between and "if" not in between, f"{name}: {fn} may leave a wait without a warp barrier"
    assert seen >= 1
