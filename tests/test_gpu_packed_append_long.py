"""gqa_packed_rope_append over many tokens, which are streamed through shared memory: rows of one
part and of several, every head dim, with and without norms, cache and queries, in place, and
device contents that it has to refuse.  Against plain 64-bit forms."""
import pytest
import torch

import global_causal_gqa_gb300 as gqa
import gpu_utils as gu
import packed_utils as pu
from test_gpu_packed import _gen, _randn, _table

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


def _bound(x, d):
    """One rounding to bf16, the table's and the products' fp32 roundings before it: a pair's two
    products are at most its length, the norm's sum of d squares adds d 2^-24 and its inverse
    root 4 of them."""
    h = x.abs()
    pair = torch.cat([h[..., :d // 2] + h[..., d // 2:]] * 2, -1)
    return pu.BF16 * h + (20 + d) * pu.FP32 * pair * 1.5


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 1, 1), (64, 5, 5), (128, 64, 8), (128, 33, 3), (128, 7, 1),
                                      (256, 16, 8), (256, 3, 1), (512, 9, 2), (512, 32, 8)])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("page,t,past", [(16, [400, 0, 1, 250, 3], [0, 9, 100, 17, 40]),
                                         (128, [609], [1])])
def test_append_long(d, Hq, Hkv, norm, page, t, past):
    gen = _gen(801 + d + Hq)
    eps, total = 1e-6, sum(t) + 3
    cu = pu.cu_of(t, 2)
    s = [a + b for a, b in zip(t, past)]
    qkv = _randn(gen, total, (Hq + 2 * Hkv) * d)
    row = qkv.shape[1]
    q, k, v = qkv.split([Hq * d, Hkv * d, Hkv * d], 1)
    gq = (1 + 0.1 * torch.randn(d, generator=gen)).cuda() if norm else None
    gk = (1 + 0.1 * torch.randn(d, generator=gen)).cuda() if norm else None
    kp, vp, table = pu.pools(len(t), s, Hkv, page, d, gen, fill=-3.0)
    lens, tab = pu.i32(s), _table(d, max(s))
    cache = gqa.make_paged_kv(kp, vp, table, lens)
    qo = torch.full((total, Hq, d), -7.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((total, Hkv, d), -7.0, dtype=torch.bfloat16, device="cuda")
    gqa.gqa_packed_rope_append(q, row, k, row, v, row, pu.i32(cu), len(t), total, Hq, Hkv, d, gq, gk,
                               eps, tab, max(s), qo, ko, cache)
    assert pu.status() == 0
    pos = torch.tensor([p + i for n, p in zip(t, past) for i in range(n)], device="cuda")
    seq = torch.tensor([i for i, n in enumerate(t) for _ in range(n)], device="cuda")
    r = slice(cu[0], cu[-1])
    rq = pu.rope64(q.reshape(total, Hq, d)[r], pos, 1e4, gq, eps)
    rk = pu.rope64(k.reshape(total, Hkv, d)[r], pos, 1e4, gk, eps)
    pu.check(qo[r], rq, _bound(rq, d), "q_out")
    pu.check(ko[r], rk, _bound(rk, d), "k_out")
    for x in (qo, ko):
        assert (x[:cu[0]] == -7).all() and (x[cu[-1]:] == -7).all()
    want_k, want_v = torch.full_like(kp, -3.0), torch.full_like(vp, -3.0)
    pg = table[seq, pos // page].long()
    want_k[pg, :, pos % page] = ko[r]
    want_v[pg, :, pos % page] = v.reshape(total, Hkv, d)[r]
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)


@pytest.mark.parametrize("total", [608, 609, 5000])
def test_append_long_equals_its_parts(total):
    """The same bits as calls of a few tokens each, and in place."""
    d, Hq, Hkv = 128, 24, 4
    q, k = _randn(_gen(811), total, Hq, d), _randn(_gen(812), total, Hkv, d)
    g, tab = torch.rand(d, generator=_gen(813)).cuda(), _table(d, total)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    for a in range(0, total, 500):
        # a step of its own: positions go on from `a`, so its table starts there
        n = min(500, total - a)
        gqa.gqa_packed_rope_append(q[a:], Hq * d, k[a:], Hkv * d, None, 0, pu.i32([0, n]), 1, n, Hq,
                                   Hkv, d, g, None, 1e-5, tab[a * d:], total - a, qo[a:], ko[a:], None)
    gqa.gqa_packed_rope_append(q, Hq * d, k, Hkv * d, None, 0, pu.i32([0, total]), 1, total, Hq, Hkv, d,
                               g, None, 1e-5, tab, total, q, k, None)
    assert pu.status() == 0
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_append_long_keys_alone():
    total, Hkv, d = 700, 2, 128
    k, v = _randn(_gen(821), total, Hkv, d), _randn(_gen(822), total, Hkv, d)
    kp, vp, table = pu.pools(1, [total], Hkv, 16, d, _gen(823), fill=0.0)
    tab, lens = _table(d, total), pu.i32([total])
    gqa.gqa_packed_rope_append(None, 0, k, Hkv * d, v, Hkv * d, pu.i32([0, total]), 1, total, 0, Hkv, d,
                               None, None, 0.0, tab, total, None, None,
                               gqa.make_paged_kv(kp, vp, table, lens))
    assert pu.status() == 0
    j = torch.arange(total, device="cuda")
    pg = table[0, j // 16].long()
    assert torch.equal(vp[pg, :, j % 16], v)
    want = pu.rope64(k, j, 1e4)
    pu.check(kp[pg, :, j % 16], want, _bound(want, d), "keys")


@pytest.mark.parametrize("what,code", [("page", -1), ("table", -8), ("lens", -1), ("pages", -4),
                                       ("offsets", -1)])
def test_append_long_bad_device_contents(what, code):
    """Flagged and left out; what is sound of the batch is written."""
    t, s, d, page = [300, 400], [310, 450], 64, 16
    total, cu = 700, [0, 300, 700]
    k = _randn(_gen(831), total, d)
    kp, vp, table = pu.pools(2, s, 1, page, d, _gen(832), fill=0.0)
    good, n_tab = table.clone(), 512
    tab, rows = _table(d, n_tab), [(0, i) for i in range(300)] + [(1, i) for i in range(400)]
    if what == "page":
        table[1, 10] = kp.shape[0]
        rows = [(a, i) for a, i in rows if a == 0 or (50 + i) // page != 10]
    elif what == "table":
        n_tab = 400
        rows = [(a, i) for a, i in rows if a == 0 or 50 + i < 400]
    elif what == "lens":
        s = [310, 399]
        rows = rows[:300]
    elif what == "pages":
        s = [310, 16 * table.shape[1] + 1]
        rows = rows[:300]
    else:
        cu = [0, 300, 701]
        rows = rows[:300]
    lens = pu.i32(s)
    gqa.gqa_packed_rope_append(None, 0, k, d, k, d, pu.i32(cu), 2, total, 0, 1, d, None, None, 0.0, tab,
                               n_tab, None, None, gqa.make_paged_kv(kp, vp, table, lens))
    assert pu.status() == code
    want = torch.zeros_like(vp)
    seq = torch.tensor([a for a, _ in rows], device="cuda")
    i = torch.tensor([b for _, b in rows], device="cuda")
    pos = i + torch.where(seq == 0, 10, 50)
    want[good[seq, pos // page].long(), 0, pos % page] = k[i + 300 * seq]
    assert torch.equal(vp, want)
