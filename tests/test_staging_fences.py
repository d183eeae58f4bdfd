"""Static check of the kernels that stage outputs in shared memory (no GPU needed).

A staging buffer is written by ordinary stores and then touched by the async proxy: a TMA
store reads it, or, where it is a slot of a load ring, a TMA load refills it.  A barrier alone
does not order the two, so a thread that arrives on a `staged` barrier must have executed
`fence_proxy_async_smem()` since its last store, whichever branches it took: the fence stands in
the arrival's own block, behind everything that writes the buffer."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "global_causal_gqa_gb300", "csrc")
FENCE = "fence_proxy_async_smem();"


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def _unfenced(code):
    """The arrivals on `staged` without a fence of their own block directly before them, but for
    statements that store nothing."""
    bad = []
    for m in re.finditer(r"mbar_arrive(_cnt)?\(&bars->staged", code):
        # the text of the arrival's own block before it, inner blocks left out
        own, depth = [], 0
        for c in reversed(code[:m.start()]):
            if c == "}":
                depth += 1
                own.append("\0")      # an inner block ended here
            elif c == "{":
                if depth == 0:
                    break
                depth -= 1
            elif depth == 0:
                own.append(c)
        own = "".join(reversed(own))
        at = own.rfind(FENCE)
        # (`if (...) fence;` would be no fence of the block itself)
        if at < 0 or "\0" in own[at:] or not re.search(r"[;\0{]\s*$|^\s*$", own[:at]):
            bad.append(code[:m.start()].count("\n") + 1)
    return bad


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith(".cu")))
def test_staged_outputs_are_fenced_on_every_path(name):
    assert _unfenced(_code(name)) == []


@pytest.mark.parametrize("block,ok", [
    ("x[0] = a; fence_proxy_async_smem(); mbar_arrive(&bars->staged);", True),
    ("if (w) { y(); } else { z(); } fence_proxy_async_smem(); mbar_arrive(&bars->staged[i]);", True),
    ("if (w) { fence_proxy_async_smem(); } else { z(); } mbar_arrive(&bars->staged);", False),
    ("if (w) fence_proxy_async_smem(); mbar_arrive(&bars->staged);", False),
    ("fence_proxy_async_smem(); if (w) { x[0] = a; } mbar_arrive(&bars->staged);", False),
    ("x[0] = a; mbar_arrive(&bars->staged);", False),
])
def test_the_check_itself(block, ok):
    assert (_unfenced("void f() { " + block + " }") == []) == ok
