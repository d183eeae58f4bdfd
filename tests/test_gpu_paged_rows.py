"""gqa_attn_paged with 17 to 32 rows (new tokens x heads of a KV group) per sequence, the fewest
that leave the streaming kernel for the tiles, next to sequences with fewer."""
import math

import pytest
import torch

import gpu_utils as gu
import packed_utils as pu
from test_gpu_packed import Paged, _paged

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


@pytest.mark.parametrize("Hq,Hkv,t", [(32, 1, [1, 1, 0, 1, 1]), (17, 1, [1, 1, 1, 1, 1]),
                                      (64, 2, [1, 0, 1, 1, 1]), (16, 2, [4, 1, 3, 2, 0]),
                                      (7, 1, [4, 4, 1, 0, 3]), (3, 3, [32, 17, 16, 1, 31]),
                                      (50, 2, [1, 1, 1, 1, 1]), (8, 4, [16, 8, 9, 1, 15]),
                                      (11, 1, [2, 1, 2, 2, 1])])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("window", [0, 1, 70])
def test_rows(Hq, Hkv, t, page, window):
    s = [t[0], 137 + t[1], 64 + t[2], 300 + t[3], 63 + t[4]]
    _paged(t, s, Hq, Hkv, page, window, 900 + Hq + page, first=1, behind=2)


@pytest.mark.parametrize("t,s", [([4], [9001]), ([4, 1, 3, 2], [700, 3000, 65, 1500]),
                                 ([2] * 90, [1 + (37 * i) % 900 + 2 for i in range(90)])])
@pytest.mark.parametrize("window", [0, 600])
def test_rows_split_over_chunks(t, s, window):
    p = _paged(t, s, 16, 2, 64, window, 930 + len(t), max_q=4)
    o, L = p.o.clone(), p.L.clone()
    p.ws.fill_(math.nan)
    p.run(window)
    assert torch.equal(p.o, o) and torch.equal(p.L, L)


def test_rows_in_levels():
    """Long sequences of 32 rows, cut into levels of chunks."""
    s, t = [26000, 31000, 3, 24000, 9, 29000, 100, 50100], [4, 2, 3, 4, 0, 1, 4, 3]
    p = Paged(t, s, 64, 8, 64, 940)
    p.run()
    assert pu.status() == 0
    p.check()


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_hidden_values_do_not_leak(window, bad):
    """A non-finite value in the newest token: only the last query sees it."""
    p = Paged([4, 4], [300, 90], 8, 1, 16, 950)
    for i, n in enumerate(p.s):
        pg = p.table[i, (n - 1) // 16].long()
        p.vp[pg, :, (n - 1) % 16, 5] = bad
        p.v[i][n - 1, :, 5] = bad
    p.run(window)
    assert pu.status() == 0
    o = p.out()
    for i in range(2):
        a, b = p.cu[i], p.cu[i + 1]
        assert not torch.isfinite(o[b - 1, :, 5]).any()
        clean = p.v[i].clone()
        clean[-1, :, 5] = 0
        ro, _, bo, _ = pu.attention64(p.q[a:b], p.k[i], clean, window, 128 ** -0.5)
        pu.check(o[a:b - 1], ro[:-1], bo[:-1], "rows that do not see it")
        keep = [c for c in range(128) if c != 5]
        pu.check(o[b - 1][:, keep], ro[-1][:, keep], bo[-1][:, keep], "other dims of the last row")


@pytest.mark.parametrize("bad", [-1, None, 2 ** 31 - 1])
def test_rows_bad_page(bad):
    p = Paged([4, 3], [200, 90], 8, 1, 16, 960)
    p.table[0, 2] = p.kp.shape[0] if bad is None else bad
    p.run()
    assert pu.status() == -1
    o = p.out()
    ro, _, bo, _ = pu.attention64(p.q[4:7], p.k[1], p.v[1], 0, 128 ** -0.5)
    pu.check(o[4:7], ro, bo, "the sound sequence")
    k, v = p.k[0].clone(), p.v[0].clone()
    k[32:48], v[32:48] = 0, 0          # zeros are read instead
    ro, _, bo, _ = pu.attention64(p.q[:4], k, v, 0, 128 ** -0.5)
    pu.check(o[:4], ro, bo, "the other one")
