"""Batches whose tiles are nearly all ragged (fewer tokens than a tile has): each one's output
leaves through a ring slot that the next item's keys or values then take.  Every item is checked
against the plain 64-bit form, and repeated runs give the same bits."""
import math

import pytest
import torch

import gpu_utils as gu
import packed_utils as pu
from test_gpu_packed import Paged, _check_packed, _packed

pytestmark = pytest.mark.gpu

# with 8 heads to a KV head a tile has 16 tokens and an item two tiles
LENS = [1 + (11 * i) % 31 for i in range(240)]


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


def test_ragged_prompts():
    _check_packed(LENS, 32, 4, 0, 301, first=1, behind=3)


def test_ragged_prompts_same_bits():
    a = _packed(LENS, 32, 4, 9, 302)
    for _ in range(4):
        b = _packed(LENS, 32, 4, 9, 302)
        assert torch.equal(a[4], b[4]) and torch.equal(a[5], b[5])


@pytest.mark.parametrize("page", [16, 128])
def test_ragged_chunks(page):
    """Chunks of 3 to 31 tokens over 0 to 290 older ones."""
    t = [3 + n % 29 for n in LENS]
    s = [a + (37 * i) % 291 for i, a in enumerate(t)]
    p = Paged(t, s, 32, 4, page, 303, behind=2)
    p.run()
    assert pu.status() == 0
    p.check()
    o, L = p.o.clone(), p.L.clone()
    for _ in range(3):
        p.ws.fill_(math.nan)
        p.run()
        assert torch.equal(p.o, o) and torch.equal(p.L, L)
    assert pu.status() == 0
