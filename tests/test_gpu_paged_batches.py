"""Large batches over the paged cache: keys cut into levels of chunks that the SMs claim, the
same bounds with little behind them, and the look-up of a token among many sequences.  Against
plain 64-bit forms."""
import pytest
import torch

import global_causal_gqa_gb300 as gqa
import gpu_utils as gu
import packed_utils as pu
from test_gpu_packed import D, Paged, _gen, _randn, _table

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


# 64 keys make a unit and 152 * 128 = 19456 units a batch that is cut into levels: these are
# 20056 of (sequence, KV head), 64 pairs of them
LONG = [26000, 31000, 3, 24000, 9, 29000, 100, 50100]


@pytest.mark.parametrize("Hq,t", [(8, [1, 1, 1, 1, 0, 1, 1, 1]),      # 1 row of each KV head
                                  (32, [4, 1, 3, 2, 0, 4, 4, 1]),    # 16 rows
                                  (64, [1, 1, 0, 1, 1, 1, 1, 1])])   # 8 rows
def test_levels_of_chunks(Hq, t):
    """Long sequences, the partials of each merged over many chunks, and the same bits again."""
    assert sum(-(-n // 64) for n, a in zip(LONG, t) if a) * 8 >= 152 * 128
    p = Paged(t, LONG, Hq, 8, 64, 700 + Hq, max_q=4 if Hq == 32 else 1, first=2, behind=1)
    p.run()
    assert pu.status() == 0
    p.check()
    o, L = p.o.clone(), p.L.clone()
    for _ in range(3):
        p.ws.fill_(float("nan"))
        p.run()
        assert torch.equal(p.o, o) and torch.equal(p.L, L)
    assert pu.status() == 0


@pytest.mark.parametrize("s", [[700, 31, 5, 64, 0, 65, 129, 1], [0] * 8, [1] * 8, [9000] * 8])
def test_bounds_of_a_large_batch_over_a_small_one(s):
    """The host's bounds ask for levels; what the device finds does not fill them."""
    t = [min(1, n) for n in s]
    if sum(t) == 0:
        p = Paged([1] * 8, [1] * 8, 16, 8, 16, 720, max_kv=60000)
        p.cu_d.zero_()
        p.t, p.cu = [0] * 8, [0] * 9
    else:
        p = Paged(t, s, 16, 8, 16, 721 + sum(s), max_kv=60000)
    p.run()
    assert pu.status() == 0
    p.check()


def test_levels_with_a_window():
    """The window leaves fewer keys than max_kv: no levels."""
    p = Paged([1, 1, 1, 1, 1, 1, 1, 1], LONG, 16, 8, 16, 731)
    p.run(window=500)
    assert pu.status() == 0
    p.check(window=500)


def test_levels_two_streams_and_a_graph():
    """Two such calls at once, one of them a replayed graph, each with its own workspace."""
    a = Paged([1] * 8, LONG, 16, 8, 64, 741)
    b = Paged([1] * 8, LONG[::-1], 16, 8, 64, 742)
    a.run()
    b.run()
    torch.cuda.synchronize()
    want = [a.o.clone(), b.o.clone()]
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            b.run(stream=side)
    torch.cuda.synchronize()
    a.o.fill_(-7.0)
    b.o.fill_(-7.0)
    torch.cuda.synchronize()
    for _ in range(4):
        with torch.cuda.stream(side):
            g.replay()
        a.run()
    torch.cuda.synchronize()
    assert pu.status() == 0
    assert torch.equal(a.o, want[0]) and torch.equal(b.o, want[1])


@pytest.mark.parametrize("n", [33, 64, 1024, 1025, 1100, 3000])
def test_append_many_sequences(n):
    """Each token's position and page among n sequences, empty ones between them."""
    t = [(0, 1, 1, 2, 0, 0, 3)[i * i % 7] for i in range(n)]
    s = [a + (5 * i) % 29 if a else 0 for i, a in enumerate(t)]
    d, total, cu = 64, sum(t) + 3, pu.cu_of(t, 2)
    k, v = _randn(_gen(751), total, d), _randn(_gen(752), total, d)
    kp, vp, table = pu.pools(n, s, 1, 16, d, _gen(753), fill=-3.0)
    lens, tab = pu.i32(s), _table(d, 32)
    q = _randn(_gen(754), total, d)
    qo = torch.full_like(q, -7.0)
    gqa.gqa_packed_rope_append(q, d, k, d, v, d, pu.i32(cu), n, total, 1, 1, d, None, None, 0.0, tab,
                               32, qo, None, gqa.make_paged_kv(kp, vp, table, lens))
    assert pu.status() == 0
    pos = torch.tensor([b - a + i for a, b in zip(t, s) for i in range(a)], device="cuda")
    seq = torch.tensor([i for i, a in enumerate(t) for _ in range(a)], device="cuda")
    r = slice(cu[0], cu[-1])
    want = pu.rope64(q[r][:, None], pos, 1e4)[:, 0]
    # one rounding to bf16; the table's and the two products' fp32 roundings: 8 of a pair's length
    h = want.abs()
    pair = torch.cat([h[:, :d // 2] + h[:, d // 2:]] * 2, -1)
    pu.check(qo[r], want, pu.BF16 * h + 16 * pu.FP32 * 1.5 * pair, "q_out")
    assert (qo[:cu[0]] == -7).all() and (qo[cu[-1]:] == -7).all()
    want_v = torch.full_like(vp, -3.0)
    want_v[table[seq, pos // 16].long(), 0, pos % 16] = v[r]
    assert torch.equal(vp, want_v)


def test_captured_levels_follow_the_lengths():
    """One captured call over lengths that fill the levels, then some that do not, none, and the
    first ones again."""
    p = Paged([1] * 8, LONG, 16, 8, 64, 761, max_kv=60000)
    p.run()
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            p.run(stream=side)
    torch.cuda.synchronize()
    full = (p.s, p.k, p.v)
    for cut in (1, 40, 1, 3000, 7, 1):
        p.s = [max(1, n // cut) for n in full[0]]
        p.k, p.v = [x[:n] for x, n in zip(full[1], p.s)], [x[:n] for x, n in zip(full[2], p.s)]
        p.s_d.copy_(pu.i32(p.s))
        p.o.fill_(-7.0)
        p.L.fill_(-7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert pu.status() == 0
        p.check()


@pytest.mark.parametrize("place", [0, 39])
def test_one_long_sequence_among_short_ones(place):
    """Enough keys for levels, but nearly all of them of one pair: a chunk per SM."""
    s = [1 + (17 * i) % 150 for i in range(40)]
    s[place] = 1250000
    assert -(-s[place] // 64) >= 152 * 128
    p = Paged([1] * 40, s, 8, 1, 128, 771)
    p.run()
    assert pu.status() == 0
    p.check()
    o = p.o.clone()
    p.ws.fill_(float("nan"))
    p.run()
    assert torch.equal(p.o, o)
