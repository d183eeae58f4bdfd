"""Calls of the packed and paged operators that are allowed but out of the ordinary: windows as
large as an int or negative, a gain for q or for k alone, tile kernels on two streams at once,
and a captured call with eager ones between its replays."""
import math

import pytest
import torch

import global_causal_gqa_gb300 as gqa
import gpu_utils as gu
import packed_utils as pu
from test_gpu_packed import D, Paged, _gen, _packed, _randn, _table

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (2, 2), (5, 1)])
@pytest.mark.parametrize("window", [MOST, MOST - 300, -1, -MOST])
def test_windows_that_hide_nothing_packed(Hq, Hkv, window):
    a = _packed([400, 1, 77], Hq, Hkv, 0, 611)
    b = _packed([400, 1, 77], Hq, Hkv, window, 611)
    assert torch.equal(a[4], b[4]) and torch.equal(a[5], b[5])


@pytest.mark.parametrize("t,s", [([1, 1], [137, 60]), ([1, 1], [9001, 700]), ([2, 1], [9001, 700]),
                                 ([40, 3], [200, 60]), ([40, 3], [9001, 700])])
@pytest.mark.parametrize("window", [MOST, -5])
def test_windows_that_hide_nothing_paged(t, s, window):
    p = Paged(t, s, 8, 1, 16, 612)
    p.run()
    p.check()
    o, L = p.o.clone(), p.L.clone()
    p.ws.fill_(math.nan)
    p.o.fill_(-7.0)
    p.run(window)
    assert pu.status() == 0
    p.check()
    assert torch.equal(p.o, o) and torch.equal(p.L, L)


@pytest.mark.parametrize("total", [9, 700])
@pytest.mark.parametrize("which", ["q", "k"])
def test_a_gain_for_one_of_them(total, which):
    """The other one's result is that of a call without gains."""
    Hq, Hkv = 6, 2
    q, k = _randn(_gen(621), total, Hq, D), _randn(_gen(622), total, Hkv, D)
    g, tab, cu = torch.rand(D, generator=_gen(623)).cuda(), _table(D, total), pu.i32([0, total])

    def call(gq, gk):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        gqa.gqa_packed_rope_append(q, Hq * D, k, Hkv * D, None, 0, cu, 1, total, Hq, Hkv, D, gq, gk,
                                   1e-6, tab, total, qo, ko, None)
        assert pu.status() == 0
        return qo, ko
    plain, both = call(None, None), call(g, g)
    got = call(g if which == "q" else None, g if which == "k" else None)
    for i, name in enumerate("qk"):
        assert torch.equal(got[i], (both if name == which else plain)[i])
        assert not torch.equal(both[i], plain[i])


def test_tile_kernels_on_two_streams():
    """Chunks, split and whole, and packed prompts at the same time, each with its own workspace."""
    ps = [Paged([40, 3], [9001, 700], 8, 1, 16, 631), Paged([200, 1], [900, 3000], 16, 2, 64, 632)]
    lens, Hq, Hkv = [700, 33, 260], 16, 2
    total, row = sum(lens), (Hq + 2 * Hkv) * D
    q, k, v = _randn(_gen(633), total, row).split([Hq * D, Hkv * D, Hkv * D], 1)
    o, cu = torch.empty(total, Hq, D, dtype=torch.bfloat16, device="cuda"), pu.i32(pu.cu_of(lens))

    def packed(stream):
        gqa.gqa_attn_packed(q, row, k, row, v, row, o, Hq * D, None, cu, len(lens), total, Hq, Hkv, D, 0,
                            D ** -0.5, stream)
    packed(None)
    for p in ps:
        p.run()
    torch.cuda.synchronize()
    want = [o.clone()] + [p.o.clone() for p in ps]
    ss = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(6):
        packed(ss[0])
        for p, s in zip(ps, ss[1:]):
            p.run(stream=s)
    torch.cuda.synchronize()
    assert pu.status() == 0
    for a, b in zip(want, [o] + [p.o for p in ps]):
        assert torch.equal(a, b)
    for p in ps:
        p.check()


@pytest.mark.parametrize("t,s", [([1, 1], [9001, 700]), ([40, 3], [9001, 700])])
def test_a_captured_call_between_eager_ones(t, s):
    """On one stream the same workspace serves both, whatever order they come in."""
    a, b = Paged(t, s, 8, 1, 16, 641), Paged(t, s[::-1] if t[0] == t[1] else s, 8, 1, 16, 642)
    assert a.wsb == b.wsb > 0
    b.ws = a.ws
    a.run()
    b.run()
    torch.cuda.synchronize()
    want = a.o.clone(), b.o.clone()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            a.run(stream=side)
    torch.cuda.synchronize()
    for _ in range(4):
        a.o.fill_(-7.0)
        b.o.fill_(-7.0)
        g.replay()
        b.run()
        torch.cuda.synchronize()
        assert torch.equal(a.o, want[0]) and torch.equal(b.o, want[1])
    assert pu.status() == 0
    a.check()
    b.check()
