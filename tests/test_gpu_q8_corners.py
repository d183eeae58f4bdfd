"""The 8-bit paged cache where calls differ from the ordinary: heads whose rows go in blocks, pools
in either order, one pool for both, pools far apart, no lse, captured calls that share a workspace,
offsets that contradict one another, outputs in place."""
import math

import pytest
import torch

import global_causal_gqa_gb300 as gqa
import gpu_utils as gu
import packed_utils as pu
import q8_utils as q8
from test_gpu_packed import D, _gen, _randn, _table
from test_gpu_packed_offsets import BAD, _claims
from test_gpu_q8 import PagedQ8, _paged

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


@pytest.mark.parametrize("Hq,Hkv,most", [(40, 1, 1), (24, 1, 2), (64, 2, 2), (33, 1, 1), (48, 4, 5),
                                         (9, 1, 7), (12, 1, 1), (64, 1, 1), (22, 2, 3),
                                         (24, 1, 4), (64, 4, 5), (7, 1, 13)])
@pytest.mark.parametrize("s_most,window", [(400, 0), (900, 0), (900, 130)])
def test_rows_in_blocks(Hq, Hkv, most, s_most, window):
    """9 to 96 rows: teams of two and four groups, up to three blocks, sequences with fewer rows."""
    t = [(3 * i + 1) % (most + 1) for i in range(11)]
    t[4] = most
    s = [max(n, 1 + (131 * i) % s_most) for i, n in enumerate(t)]
    _paged(t, s, Hq, Hkv, 32, window, 800 + Hq + s_most, first=1, behind=2)


@pytest.mark.parametrize("t,n", [(1, 3), (1, 930), (3, 3), (6, 3), (70, 3)])
def test_no_lse(t, n):
    p = PagedQ8([t] * n, [200] * n, 8, 1, 16, 811)
    p.run()
    o = p.o.clone()
    p.o.fill_(-7)
    gqa.gqa_attn_paged_q8(p.q, 8 * D, p.cache, p.cu_d, n, p.total, t, 200, 8, 0, D ** -0.5, p.o,
                          8 * D + 8, None, p.ws, p.wsb)
    assert pu.status() == 0 and torch.equal(p.o, o)


@pytest.mark.parametrize("t,n", [(1, 2), (1, 930), (2, 2), (7, 2)])
@pytest.mark.parametrize("how", ["values first", "one pool", "far apart"])
def test_places_of_the_pools(t, n, how):
    """Values that lie before the keys, values that are the keys, and small pools 12 GB apart."""
    p = PagedQ8([t] * n, [300 if n == 2 else 90] * n, 8, 1, 16, 812 + t)
    if how == "values first":
        both = torch.empty(2, *p.kq.shape, dtype=torch.uint8, device="cuda")
        both[0], both[1] = p.vq, p.kq
        p.vq, p.kq = both[0], both[1]
    elif how == "far apart":
        room = torch.empty(12 << 30, dtype=torch.uint8, device="cuda")
        n = p.kq.numel()
        ends = [x.reshape(p.kq.shape) for x in (room[:n], room[-n:])]
        ends[0].copy_(p.kq)
        ends[1].copy_(p.vq)
        p.kq, p.vq = ends
    else:
        p.vq = p.kq
        p.sc[..., 1] = p.sc[..., 0]
        for x in p.rows:
            x[2], x[3] = x[0], x[1]
    p.cache = q8.cache_of(p.kq, p.vq, p.sc, p.table, p.s_d)
    p.run()
    assert pu.status() == 0
    p.check(only=None if n == 2 else range(0, n, 17))


@pytest.mark.parametrize("t", [1, 3, 6, 30])
def test_captured_calls_that_share_a_workspace(t):
    """Two captured calls of different batches with one workspace, replayed in turn on one stream."""
    ps = [PagedQ8([t] * 5, [3000, 30 + 7 * i, 1000, 512, 64], 8, 2, 16, 820 + i, max_kv=4000)
          for i in range(2)]
    ps[1].ws, ps[1].wsb = ps[0].ws, ps[0].wsb
    for p in ps:
        p.run()
    torch.cuda.synchronize()
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            p.run()
        graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    for p in ps:
        p.o.fill_(-7)
        p.L.fill_(-7)
    ps[0].ws.fill_(math.nan)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert pu.status() == 0
    for p in ps:
        p.check()


@pytest.mark.parametrize("t", [2, 5])
def test_drafts_on_two_streams(t):
    ps = [PagedQ8([t] * 4, [4000, 30, 1000, 512], 8, 2, 16, 830 + i) for i in range(2)]
    ss = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s in zip(ps, ss):
            p.run(stream=s)
    torch.cuda.synchronize()
    assert pu.status() == 0
    for p in ps:
        p.check()


FEW = [[0, 3, 2, 5], [-1, 2, 4, 5], [0, 6, 20], [-5, 0, 6], [0, 6, 1], [0, 5, 2 ** 31 - 1]]


@pytest.mark.parametrize("cu,total,Hq,Hkv,max_kv",
                         [(x, 10, *y) for x in BAD for y in ((8, 8, 64), (8, 8, 600), (4, 1, 600),
                                                             (16, 1, 64))] +
                         [(x, 6, *y) for x in FEW for y in ((2, 2, 64), (2, 2, 600), (64, 64, 64))])
def test_attention_with_contradictory_offsets(cu, total, Hq, Hkv, max_kv):
    """Sound sequences are served, rows of none left, and the status word tells."""
    p = PagedQ8([1] * (len(cu) - 1), [40] * (len(cu) - 1), Hq, Hkv, 16, 840, max_kv=max_kv)
    q = _randn(_gen(841), total, Hq, D)
    o = torch.full((total, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    n_seq = len(cu) - 1
    wsb = gqa.gqa_attn_paged_q8_workspace_bytes(n_seq, total, total, max_kv, Hq, Hkv, D)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device="cuda")
    gqa.gqa_attn_paged_q8(q, Hq * D, p.cache, pu.i32(cu), n_seq, total, total, max_kv, Hq, 0,
                          D ** -0.5, o, Hq * D, None, ws, wsb)
    assert pu.status() == -1
    sound, n = _claims(cu, total)
    for i, a, b in sound:
        rows = [r for r in range(a, b) if n[r] == 1]
        if not rows:
            continue
        at = torch.tensor(rows, device="cuda")
        ro, _, bo, _ = q8.attention64(q[a:b], *p.rows[i], 0, D ** -0.5)
        pu.check(o[at], ro[at - a], bo[at - a], f"o of sequence {i}")
    for r in range(total):
        if n[r] == 0:
            assert (o[r] == 3).all()


@pytest.mark.parametrize("cu", BAD)
def test_read_and_append_with_contradictory_offsets(cu):
    """These find a row's sequence by bisection: rows of sound sequences are served where the
    offsets ascend; where they do not, the search may end at another sequence, and a row is left as
    it was unless it lies in the one found.  Never is it anything else."""
    total, n_seq = 10, len(cu) - 1
    p = PagedQ8([1] * n_seq, [40] * n_seq, 2, 2, 16, 842)
    sound, n = _claims(cu, total)
    ascend = cu == sorted(cu)
    out = torch.full((total, 2, D), 3.0, dtype=torch.bfloat16, device="cuda")
    gqa.gqa_paged_read_q8(p.cache, pu.i32(cu), n_seq, total, out, 2 * D, None, 0)
    assert pu.status() == -1
    left = torch.full((2, D), 3.0, dtype=torch.bfloat16, device="cuda")
    for r in range(total):
        may = [q8.values(*(x[40 - b + r] for x in p.rows[i][:2])).to(torch.bfloat16)
               for i, a, b in sound if a <= r < b]
        if not ascend or not may:
            may.append(left)
        assert any(torch.equal(out[r], x) for x in may), r
    k = _randn(_gen(843), total, 2 * D)
    before = p.vq.clone()
    gqa.gqa_packed_rope_append_q8(None, 0, k, 2 * D, k, 2 * D, pu.i32(cu), n_seq, total, 0, 2, D, None,
                                  None, 0.0, _table(D, 64), 64, None, None, p.cache)
    assert pu.status() == -1
    data, _ = q8.quantise(k.reshape(total, 2, D))
    claimed = torch.zeros_like(before, dtype=torch.bool)
    for i, a, b in sound:
        for r in range(a, b):
            pg, slot = q8.places(p.table, i, 16, 40 - b + r)
            claimed[pg, :, slot] = True
            new, old = (torch.equal(p.vq[pg, :, slot], x) for x in (data[r], before[pg, :, slot]))
            # (rows of two sequences go to one of them)
            assert new or (old and (n[r] > 1 or not ascend)), (i, r)
    assert torch.equal(p.vq[~claimed], before[~claimed])


@pytest.mark.parametrize("n", [40, 700])
def test_append_in_place(n):
    """q and k rotated where they lie, next to the write of the cache."""
    Hq, Hkv = 4, 2
    q, k = _randn(_gen(850), n, Hq, D), _randn(_gen(851), n, Hkv, D)
    v = _randn(_gen(852), n, Hkv, D)
    tab = _table(D, n)
    kq, vq, sc, table = q8.pools(1, [n], Hkv, 16, D, _gen(853))
    cache = q8.cache_of(kq, vq, sc, table, pu.i32([n]))
    cu = pu.i32([0, n])
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    args = (v, Hkv * D, cu, 1, n, Hq, Hkv, D, None, None, 0.0, tab, n)
    gqa.gqa_packed_rope_append_q8(q, Hq * D, k, Hkv * D, *args, qo, ko, cache)
    a = [x.clone() for x in (kq, vq, sc)]
    gqa.gqa_packed_rope_append_q8(q, Hq * D, k, Hkv * D, *args, q, k, cache)
    assert pu.status() == 0
    assert torch.equal(q, qo) and torch.equal(k, ko)
    for x, y in zip(a, (kq, vq, sc)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("t,n", [(1, 3), (1, 930), (3, 3), (6, 3)])
def test_nonfinite_queries_make_their_row_nan(bad, t, n):
    p = PagedQ8([t] * n, [60] * n, 8, 1, 16, 860)
    p.run()
    clean, L = p.out().clone(), p.L.clone()
    p.q[1, 3, 5] = bad
    p.run()
    assert pu.status() == 0
    want = clean.clone()
    want[1, 3] = math.nan
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(p.out()), nan) and torch.equal(p.out()[~nan], clean[~nan])
    assert torch.isnan(p.L[3, 1])
    p.L[3, 1] = L[3, 1]
    assert torch.equal(p.L, L)


def test_any_range_is_read():
    """Another kv_lens reads other tokens of the same pages."""
    p = PagedQ8([1, 1], [300, 100], 2, 2, 16, 870)
    lens, cu = pu.i32([210, 40]), pu.i32([0, 57, 97])
    out = torch.empty(2, 97, 2, D, dtype=torch.bfloat16, device="cuda")
    cache = q8.cache_of(p.kq, p.vq, p.sc, p.table, lens)
    gqa.gqa_paged_read_q8(cache, cu, 2, 97, out[0], 2 * D, out[1], 2 * D)
    assert pu.status() == 0
    for w in range(2):
        x = [q8.values(*r[2 * w:2 * w + 2]).to(torch.bfloat16) for r in p.rows]
        assert torch.equal(out[w], torch.cat([x[0][153:210], x[1][:40]]))

