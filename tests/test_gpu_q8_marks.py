"""NaN numbers among the last tokens' values, which only some rows see: they reach those rows' dims
and nothing of the heads and sequences that a CTA takes after them, whatever rows these have."""
import math

import pytest
import torch

import gpu_utils as gu
import packed_utils as pu
from test_gpu_q8 import PagedQ8

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


def _lens(n, least, most):
    return [least + (37 * i) % (most - least + 1) for i in range(n)]


# Tokens of every sequence with 8 heads a group: drafts whose second block of rows has 8, 16 or no
# rows next to full ones, and teams of two groups with and without rows in turn (a CTA's pairs are
# every 152nd one, 19 sequences of 8 heads apart, and its teams take them in turn).
DRAFTS = {
    "5": [5] * 40,
    "6": [6] * 40,
    "1 to 12": [1 + (5 * i) % 12 for i in range(60)],
    "1 and 4": [4 if i % 2 else 1 for i in range(60)],
    "1 and 2": [1 + (i // 38 + 1) % 2 for i in range(152)],
    "1 and 2, ragged": [1 + (7 * i) % 2 for i in range(152)],
}


@pytest.mark.parametrize("t", DRAFTS)
@pytest.mark.parametrize("s,window", [((20, 512), 0), ((20, 512), 33), ((130, 1000), 0),
                                      ((130, 1000), 140)])
def test_marks_stay_with_their_rows(t, s, window):
    """A number of one head's value at one of a sequence's new tokens, or at a key that a window
    hides from the last row, in every third sequence: all other rows keep their bits."""
    t, Hq, Hkv = DRAFTS[t], 64, 8
    p = PagedQ8(t, _lens(len(t), *s), Hq, Hkv, 16, 940 + len(t), max_kv=s[1])
    p.run(window)
    assert pu.status() == 0
    clean, L = p.out().clone(), p.L.clone()
    assert torch.isfinite(clean).all()
    want = clean.clone()
    for i in range(0, len(t), 3):
        n, a, g, dim = p.s[i], p.cu[i], i % Hkv, (29 * i) % 128
        j = n - 1 - (i // 3) % t[i]
        if window and i % 2 and n - t[i] - window >= 0:
            j = n - t[i] - window + 1            # the first row's first key
        p.vq[p.table[i, j // 16].long(), g, j % 16, dim] = 0x7f
        for r in range(t[i]):
            pos = n - t[i] + r
            if j <= pos and (not window or pos - j < window):
                want[a + r, 8 * g:8 * g + 8, dim] = math.nan
    p.run(window)
    assert pu.status() == 0
    nan = torch.isnan(want)
    got = p.out()
    wrong = (torch.isnan(got) != nan).nonzero()
    assert len(wrong) == 0, f"{len(wrong)} elements, the first {wrong[0].tolist()}"
    assert torch.equal(got[~nan], want[~nan]) and torch.equal(p.L, L)
