"""Many short 8-bit caches, a warp per pair of (sequence, KV head): lengths from one token, empty
sequences, drafts, windows, page sizes, strides, contents that are hidden or wrong, against plain
64-bit forms (of some of the sequences, others in every case)."""
import math

import pytest
import torch

import gpu_utils as gu
import packed_utils as pu
import q8_utils as q8
from test_gpu_q8 import D, PagedQ8, _paged

pytestmark = pytest.mark.gpu
N = 930      # sequences: more pairs than six per SM


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


def _some(n, seed):
    """The first and last sequences and every 13th from a place of its own."""
    return {0, 1, n - 2, n - 1, *range(seed % 13, n, 13)}


def _lens(t, most=512):
    return [max(n, 1 + (37 * i) % most) for i, n in enumerate(t)]


@pytest.mark.parametrize("Hq,Hkv,page,window", [
    (8, 1, 16, 0), (8, 1, 64, 70), (3, 1, 16, 70), (3, 1, 128, 0), (1, 1, 32, 70), (1, 1, 128, 70),
    (4, 2, 32, 0), (4, 2, 64, 0)])
def test_decode(Hq, Hkv, page, window):
    t = [0 if i % 11 == 5 else 1 for i in range(N)]
    _paged(t, _lens(t), Hq, Hkv, page, window, 700 + Hq + page, first=2, behind=3,
           only=_some(N, Hq + page // 16 + window))


@pytest.mark.parametrize("Hq,Hkv,most", [(4, 1, 2), (2, 1, 4), (1, 1, 8), (6, 2, 2)])
@pytest.mark.parametrize("window", [0, 1, 33])
def test_drafts(Hq, Hkv, most, window):
    t = [(7 * i) % (most + 1) for i in range(N)]
    _paged(t, _lens(t, 300), Hq, Hkv, 16, window, 720 + Hq + window, only=_some(N, Hq + window))


def test_several_pairs_per_warp():
    n = 4000
    t = [0 if i % 7 == 3 else 1 for i in range(n)]
    _paged(t, [1 + (13 * i) % 90 for i in range(n)], 2, 1, 32, 0, 730, only=_some(n, 5))


def test_the_longest():
    _paged([1] * 240, [512 - i % 3 for i in range(240)], 16, 4, 16, 0, 731,
           only=_some(240, 1))


@pytest.mark.parametrize("n", [152, 200])
def test_two_steps_at_most(n):
    _paged([1] * n, [1 + (7 * i) % 64 for i in range(n)], 8, 1, 16, 0, 738, max_kv=64,
           only=_some(n, 2))


def test_one_long_among_empty_ones():
    t = [0] * N
    t[417] = 1
    _paged(t, [500] * N, 8, 2, 16, 0, 732)


@pytest.mark.parametrize("how", ["byte", "number"])
@pytest.mark.parametrize("window", [0, 40])
def test_hidden_values_do_not_leak(how, window):
    """NaN values at every sequence's last token and one in the middle: rows that do not see them
    are those of the clean caches."""
    t, s = [2] * N, [200] * N
    p = PagedQ8(t, s, 4, 1, 16, 733)
    p.run(window)
    clean, L = p.out().clone(), p.L.clone()
    for j in (100, 199):
        pages = p.table[:, j // 16].long()
        if how == "byte":
            p.sc[pages, :, j % 16, 1] = 255
        else:
            p.vq[pages, :, j % 16, 77] = 0x7f
    p.run(window)
    assert pu.status() == 0
    sees = torch.ones(N, 2, dtype=torch.bool, device="cuda")
    if window:
        sees[:, 0] = False                # the first token sees 159 .. 198
    sees = sees.reshape(-1)
    want = clean.clone()
    if how == "byte":
        want[sees] = math.nan
    else:
        want[sees, :, 77] = math.nan
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(p.out()), nan)
    assert torch.equal(p.out()[~nan], want[~nan]) and torch.equal(p.L, L)


@pytest.mark.parametrize("what,code", [("page", -1), ("lens", -1), ("bound", -4)])
def test_bad_device_contents(what, code):
    """A page outside the pool reads as zeros; sequences whose numbers do not fit are left; the
    others are served."""
    p = PagedQ8([1] * N, _lens([1] * N, 300), 8, 1, 16, 734, max_kv=400)
    bad = [3, 77, N - 1]
    for i in bad:
        if what == "page":
            p.table[i, 0] = -1 if i == 3 else 2 ** 31 - 1
        elif what == "lens":
            p.s_d[i] = 0
        else:
            p.s_d[i] = 401
    p.run()
    assert pu.status() == code
    if what == "page":
        for i in bad:
            for x in p.rows[i][0], p.rows[i][2]:
                x[:16] = 0
    p.check(skip=() if what == "page" else bad, only={*bad, *_some(N, 3)})


def test_spread_and_rising_scores():
    """Values' powers of two far apart; scores that rise with every step."""
    p = PagedQ8([1] * N, [150] * N, 8, 1, 16, 735, spread=20)
    x = torch.linspace(-40, 40, 150, device="cuda", dtype=torch.float64)[:, None, None]
    for i in range(0, N, 5):
        u = p.q[i, 0].double()
        p.q[i] = p.q[i, 0]
        p.rows[i][0], p.rows[i][1] = q8.quantise(x * (u * D ** 0.5 / u.dot(u)))
        p.put(i)
    p.run()
    assert pu.status() == 0
    p.check(only=range(0, N, 8))


def test_same_bits_every_run_and_stream():
    p = PagedQ8([1] * N, _lens([1] * N), 8, 1, 16, 736)
    p.run()
    a, L = p.o.clone(), p.L.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s.cuda_stream):
        p.o.fill_(-7)
        torch.cuda.synchronize()
        p.run(stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(p.o, a) and torch.equal(p.L, L)
    assert pu.status() == 0
    p.check(only=_some(N, 7))


def test_captured():
    p = PagedQ8([1] * N, _lens([1] * N, 300), 8, 1, 16, 737, max_kv=512)
    p.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        p.run()
    torch.cuda.current_stream().wait_stream(side)
    # shorter lengths of the same caches
    for i in range(N):
        p.s[i] = max(1, p.s[i] - i % 5)
        p.rows[i] = [x[:p.s[i]] for x in p.rows[i]]
    p.s_d.copy_(pu.i32(p.s))
    p.o.fill_(-7)
    g.replay()
    torch.cuda.synchronize()
    assert pu.status() == 0
    p.check(only=_some(N, 9))
