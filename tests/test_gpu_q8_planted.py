"""Long 8-bit caches in which every unit of 64 keys has a weight of its own (planted_keys.py): the
cuts into chunks, levels, spans and their merges lose none and count none twice."""
import math

import pytest
import torch

import gpu_utils as gu
import packed_utils as pu
import planted_keys
import q8_utils as q8
from test_gpu_packed import D, _gen
from test_gpu_paged_planted import LONG
from test_gpu_q8 import PagedQ8

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


def _planted(t, s, Hq, Hkv, page, seed, window=0, **kw):
    p = PagedQ8(t, s, Hq, Hkv, page, seed, **kw)
    for i, n in enumerate(t):
        if n == 0:
            continue
        a, b = p.cu[i], p.cu[i + 1]
        p.q[a:b] = planted_keys.queries(_gen(seed + i), n, Hq, D, "cuda")
        k, v = q8.values(*p.rows[i][:2]), q8.values(*p.rows[i][2:])
        planted_keys.plant(p.q[a:b], k, v)
        p.rows[i] = [*q8.quantise(k), *q8.quantise(v)]
        p.put(i)
    p.run(window)
    assert pu.status() == 0
    p.check(window)
    return p


@pytest.mark.parametrize("Hq,t,page", [(8, [1, 1, 1, 1, 0, 1, 1, 1], 16),
                                       (32, [4, 1, 3, 2, 0, 4, 4, 1], 64),
                                       (64, [1, 1, 0, 1, 1, 1, 1, 1], 128),
                                       (64, [4, 2, 3, 4, 0, 1, 4, 3], 32)])
def test_levels(Hq, t, page):
    """(Twice the keys that make levels of a bf16 cache: stages hold twice as many.)"""
    p = _planted(t, [2 * n for n in LONG], Hq, 8, page, 500 + Hq, max_q=max(t), first=2, behind=1)
    o = p.o.clone()
    p.ws.fill_(math.nan)
    p.run()
    assert torch.equal(p.o, o)


@pytest.mark.parametrize("Hq,place", [(1, 39), (8, 21), (16, 0)])
def test_one_long_sequence_among_short_ones(Hq, place):
    s = [1 + (17 * i) % 150 for i in range(40)]
    s[place] = 400000 if Hq == 1 else 1250000
    _planted([1] * 40, s, Hq, 1, 128, 520 + Hq)


@pytest.mark.parametrize("Hq,Hkv,t,s", [(8, 2, [1], [9001]), (8, 1, [2], [60000]),
                                        (8, 8, [1] * 6, [3000, 10, 700, 1, 90, 2500]),
                                        (64, 8, [1] * 5, [513, 9000, 577, 4097, 100]),
                                        (16, 2, [1] * 60, [600 + 97 * i for i in range(60)])])
@pytest.mark.parametrize("window", [0, 2048])
def test_a_chunk_per_sm(Hq, Hkv, t, s, window):
    _planted(t, s, Hq, Hkv, 32, 540 + Hq, window=window)


@pytest.mark.parametrize("Hq,Hkv,t,s", [
    (8, 1, [3], [9001]), (8, 1, [6], [9001]), (8, 1, [40], [9001]), (8, 1, [200], [30000]),
    (64, 8, [4, 2, 3, 4, 0, 1, 4, 3], LONG), (64, 8, [150, 1, 20], [9000, 3000, 12000]),
    (16, 2, [300, 1, 77, 5], [3000, 10, 700, 20000]), (2, 2, [130, 260], [5000, 7000])])
@pytest.mark.parametrize("window", [0, 2048])
def test_tiles_and_spans(Hq, Hkv, t, s, window):
    _planted(t, s, Hq, Hkv, 64, 560 + Hq, window=window, behind=2)


@pytest.mark.parametrize("t", [[1, 1, 1], [3, 1, 4], [40, 1, 7]])
def test_loose_bounds(t):
    _planted(t, [9000, 40, 3000], 8, 2, 16, 580, max_q=max(t) + 1, max_kv=200000)
