"""The sources that derive addresses from device-side data (descriptors, offsets, lengths, page
tables) carry the debug build's index checks (no GPU needed), each with a site of its own
within its kernel's code."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "global_causal_gqa_gb300", "csrc")


def _text(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name,least", [("kv.cu", 1), ("qknorm.cu", 1), ("chunk.cu", 3),
                                        ("decode.cu", 6), ("packed_append.cu", 4),
                                        ("packed_prefill.cu", 8), ("paged_decode.cu", 8)])
def test_sources_with_checks(name, least):
    assert _text(name).count("GQA_IN_BOUNDS(") >= least


def test_sites_of_the_packed_kernels():
    """Sites of one kernel code (6: append, 7: prefill, 8: decode) mean one kind of access each,
    and fit the 20 bits below the code's flag."""
    used = {}
    for name in ("kv.cu", "qknorm.cu", "chunk.cu"):
        used[name] = {int(x) for x in re.findall(r"\(kDiagCache << 24\) \| (\d+)", _text(name))}
    used["packed_append.cu"] = {int(x) for x in re.findall(r"kSite \| (\d+)",
                                                           _text("packed_append.cu"))}
    names = sorted(used)
    for i, a in enumerate(names):
        assert used[a] and max(used[a]) < 1 << 16
        for b in names[i + 1:]:
            assert not used[a] & used[b], (a, b)
