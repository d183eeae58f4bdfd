"""Packed prompts and the paged cache on the GPU: gqa_attn_packed, gqa_packed_rope_append and
gqa_attn_paged against plain 64-bit forms, at the sizes, strides, masks and contents where
they can go wrong."""
import math

import pytest
import torch

import global_causal_gqa_gb300 as gqa
import gpu_utils as gu
import packed_utils as pu

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen).to(torch.bfloat16).cuda()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ---- packed prompts ---------------------------------------------------------------------------

def _packed(lens, Hq, Hkv, window, seed, first=0, behind=0, edit=None, scale=None, lse=True):
    """Runs one call on a fused qkv tensor with rows before the first and behind the last
    sequence that hold NaN; returns what a test compares."""
    gen = _gen(seed)
    scale = D ** -0.5 if scale is None else scale
    cu = pu.cu_of(lens, first)
    total = cu[-1] + behind
    qkv = _randn(gen, total, (Hq + 2 * Hkv) * D)
    qkv[:first] = math.nan
    qkv[cu[-1]:] = math.nan
    row = qkv.shape[1]
    q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], 1)
    if edit:
        edit(q, k, v, cu)
    # the output rows are slices of wider ones, whose other columns must stay as they were
    wide = torch.full((total, Hq * D + 8), -7.0, dtype=torch.bfloat16, device="cuda")
    L = torch.full((Hq, total), -7.0, device="cuda") if lse else None
    gqa.gqa_attn_packed(q, row, k, row, v, row, wide, Hq * D + 8, L, pu.i32(cu), len(lens), total,
                        Hq, Hkv, D, window, scale)
    st = pu.status()
    assert st == 0, gqa.STATUS_NAMES.get(st, st)
    assert (wide[:, Hq * D:] == -7).all()
    o = wide[:, :Hq * D].reshape(total, Hq, D)
    for rows in (slice(0, first), slice(cu[-1], total)):
        assert (o[rows] == -7).all() and (L is None or (L[:, rows] == -7).all())
    return (q.reshape(total, Hq, D), k.reshape(total, Hkv, D), v.reshape(total, Hkv, D), cu, o, L,
            scale)


def _check_packed(lens, Hq, Hkv, window, seed, **kw):
    q, k, v, cu, o, L, scale = _packed(lens, Hq, Hkv, window, seed, **kw)
    for i, n in enumerate(lens):
        if n == 0:
            continue
        a, b = cu[i], cu[i + 1]
        ro, rl, bo, bl = pu.attention64(q[a:b], k[a:b], v[a:b], window, scale)
        pu.check(o[a:b], ro, bo, f"o of sequence {i} ({n})")
        if L is not None:
            pu.check(L[:, a:b], rl, bl, f"lse of sequence {i} ({n})")


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (4, 4), (6, 2), (5, 1), (16, 1), (14, 2), (64, 1)])
@pytest.mark.parametrize("lens", [[1], [17], [128], [129, 0, 1, 127, 300]])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_packed_shapes(lens, Hq, Hkv, window):
    _check_packed(lens, Hq, Hkv, window, 11 + Hq + len(lens) + window)


@pytest.mark.parametrize("window", [0, 2, 63, 128, 129, 500, 1000000])
def test_packed_longer(window):
    _check_packed([777, 1500, 3, 1024, 0, 640], 16, 2, window, 31 + window, first=5, behind=9)


def test_packed_many_sequences():
    lens = [(7 * i) % 41 for i in range(300)]
    _check_packed(lens, 8, 1, 0, 41, behind=2)


def test_packed_plamo_heads_and_no_lse():
    _check_packed([513, 2300], 64, 8, 2048, 43, lse=False)


def test_packed_all_empty():
    o = torch.full((4, 2, D), 3.0, dtype=torch.bfloat16, device="cuda")
    q = _randn(_gen(1), 4, 4 * D)
    gqa.gqa_attn_packed(q, 4 * D, q, 4 * D, q, 4 * D, o, 2 * D, None, pu.i32([2, 2, 2]), 2, 4, 2,
                        2, D, 0, 1.0)
    assert pu.status() == 0 and (o == 3).all()


@pytest.mark.parametrize("scale", [1e-3, 4.0])
def test_packed_scales(scale):
    """Flat weights, and weights of which a few carry all."""
    _check_packed([400, 31], 8, 2, 0, 47, scale=scale)


def test_packed_rising_scores():
    """The row maximum grows with every key tile: the running rescale is taken each time."""
    def edit(q, k, v, cu):
        n = cu[-1]
        k.copy_((k.float() * torch.linspace(0.05, 6.0, n, device="cuda")[:, None]).to(k.dtype))
    _check_packed([1100], 8, 2, 0, 53, edit=edit)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (2, 2)])
def test_packed_hidden_values_do_not_leak(bad, window, Hq, Hkv):
    """Non-finite keys and values at some tokens: rows that do not see them are exactly those
    of the clean inputs; rows that do are non-finite where the definition says so."""
    lens, at = [300, 200], (150, 151, 260)     # tokens of the first sequence
    clean = _packed(lens, Hq, Hkv, window, 59)

    def edit(q, k, v, cu):
        for t in at:
            v[t] = bad
    dirty = _packed(lens, Hq, Hkv, window, 59, edit=edit)
    n = lens[0]
    i = torch.arange(n, device="cuda")
    sees = torch.zeros(n, dtype=torch.bool, device="cuda")
    for t in at:
        sees |= (i >= t) & ((i - t < window) if window else torch.ones_like(sees))
    o0, o1 = clean[4], dirty[4]
    assert torch.equal(o1[:n][~sees], o0[:n][~sees])
    assert torch.equal(o1[n:], o0[n:])
    assert torch.equal(dirty[5], clean[5])     # lse does not look at values
    assert not torch.isfinite(o1[:n][sees]).any()
    if bad != bad:
        assert torch.isnan(o1[:n][sees]).all()
    else:
        assert (o1[:n][sees] == bad).all()


def test_packed_single_nonfinite_element():
    """One infinite element of one value: only that dimension of the rows that see it."""
    def edit(q, k, v, cu):
        v[40, 77] = math.inf
    clean = _packed([64], 4, 1, 0, 61)
    dirty = _packed([64], 4, 1, 0, 61, edit=edit)
    o0, o1 = clean[4], dirty[4]
    want = o0.clone()
    want[40:, :, 77] = math.inf
    assert torch.equal(o1, want)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_packed_hidden_keys_do_not_leak(bad):
    def edit(q, k, v, cu):
        k[100] = bad
    clean = _packed([180, 70], 8, 2, 0, 67)
    dirty = _packed([180, 70], 8, 2, 0, 67, edit=edit)
    assert torch.equal(dirty[4][:100], clean[4][:100])
    assert torch.equal(dirty[4][180:], clean[4][180:])
    assert torch.equal(dirty[5][:, :100], clean[5][:, :100])


def test_packed_same_bits_every_run_and_stream():
    a = _packed([700, 33], 16, 2, 0, 71)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = _packed([700, 33], 16, 2, 0, 71)
    s.synchronize()
    assert torch.equal(a[4], b[4]) and torch.equal(a[5], b[5])


@pytest.mark.parametrize("cu", [[0, 5, 3, 9], [-1, 4, 6, 9], [0, 4, 6, 13]])
def test_packed_inconsistent_offsets(cu):
    """Offsets that decrease, are negative or pass the rows: flagged, and only sequences with
    sound offsets are written."""
    Hq, total = 2, 10
    q = _randn(_gen(73), total, 4 * D)
    o = torch.full((total, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    gqa.gqa_attn_packed(q, 4 * D, q, 4 * D, q, 4 * D, o, Hq * D, None, pu.i32(cu), 3, total, Hq,
                        1, D, 0, 1.0)
    assert pu.status() == -1
    assert pu.status() == 0


# ---- norm, RoPE, append -------------------------------------------------------------------------

def _table(d, n, theta=1e4, amp=1.0):
    w = gqa.gqa_rope_inv_freq(d, theta)
    t = torch.empty(n * d, dtype=torch.float32, device="cuda")
    gqa.gqa_rope_table_build(t, w, d, amp, n)
    return t


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("Hq,Hkv,t,past", [(8, 2, [1], [137]), (5, 5, [3, 0, 40], [0, 7, 16]),
                                           (64, 8, [1] * 9, [0, 15, 16, 17, 31, 5, 6, 100, 127]),
                                           (3, 1, [70, 259], [1, 0])])
def test_append(d, page, norm, Hq, Hkv, t, past):
    gen = _gen(81 + d + Hq)
    eps, amp, total = 1e-6, 1.25, sum(t) + 2
    cu = pu.cu_of(t, 1)
    s = [a + b for a, b in zip(t, past)]
    qkv = _randn(gen, total, (Hq + 2 * Hkv) * d)
    row = qkv.shape[1]
    q, k, v = qkv.split([Hq * d, Hkv * d, Hkv * d], 1)
    gq = (1 + 0.1 * torch.randn(d, generator=gen)).cuda() if norm else None
    gk = (1 + 0.1 * torch.randn(d, generator=gen)).cuda() if norm else None
    kp, vp, table = pu.pools(len(t), s, Hkv, page, d, gen, fill=-3.0)
    lens = pu.i32(s)      # the struct holds addresses only: the tensor has to live on
    cache = gqa.make_paged_kv(kp, vp, table, lens)
    qo = torch.full((total, Hq, d), -7.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((total, Hkv, d), -7.0, dtype=torch.bfloat16, device="cuda")
    tab = _table(d, max(s), amp=amp)
    gqa.gqa_packed_rope_append(q, row, k, row, v, row, pu.i32(cu), len(t), total, Hq, Hkv, d, gq,
                               gk, eps, tab, max(s), qo, ko, cache)
    assert pu.status() == 0
    pos = torch.tensor([p + i for n, p in zip(t, past) for i in range(n)], device="cuda")
    r = slice(cu[0], cu[-1])
    rq = pu.rope64(q.reshape(total, Hq, d)[r], pos, 1e4, gq, eps, amp)
    rk = pu.rope64(k.reshape(total, Hkv, d)[r], pos, 1e4, gk, eps, amp)
    # one rounding to bf16, the table's and the products' fp32 roundings before it: a pair's
    # two products are at most its length, and the norm's sum of d squares adds d 2^-24
    def bound(x):
        h = x.abs()
        pair = torch.cat([h[..., :d // 2] + h[..., d // 2:]] * 2, -1)
        return pu.BF16 * h + (16 + d) * pu.FP32 * pair * 1.5
    pu.check(qo[r], rq, bound(rq), "q_out")
    pu.check(ko[r], rk, bound(rk), "k_out")
    assert (qo[:cu[0]] == -7).all() and (qo[cu[-1]:] == -7).all()
    want_k, want_v = torch.full_like(kp, -3.0), torch.full_like(vp, -3.0)
    at = cu[0]
    for i, (n, p0) in enumerate(zip(t, past)):
        j = torch.arange(p0, p0 + n, device="cuda")
        pg = table[i].long()[(j // page)]
        want_k[pg, :, j % page] = ko[at:at + n]
        want_v[pg, :, j % page] = v.reshape(total, Hkv, d)[at:at + n]
        at += n
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)


def test_append_without_a_cache_and_in_place():
    """Prompts from position 0, q and k rotated in place."""
    Hq, Hkv, t = 4, 2, [5, 33]
    total, cu = 38, pu.cu_of(t)
    q, k = _randn(_gen(91), total, Hq, D), _randn(_gen(92), total, Hkv, D)
    q0, k0 = q.clone(), k.clone()
    tab = _table(D, 33)
    gqa.gqa_packed_rope_append(q, Hq * D, k, Hkv * D, None, 0, pu.i32(cu), 2, total, Hq, Hkv, D,
                               None, None, 0.0, tab, 33, q, k, None)
    assert pu.status() == 0
    for i, n in enumerate(t):
        for x, x0, H in ((q, q0, Hq), (k, k0, Hkv)):
            y = torch.empty(1, H, n, D, dtype=torch.bfloat16, device="cuda")
            xin = x0[cu[i]:cu[i + 1]].transpose(0, 1).contiguous()
            gqa.gqa_rope_apply(xin, y, 1, H, n, D, 0, tab, 33)
            assert torch.equal(x[cu[i]:cu[i + 1]], y[0].transpose(0, 1))


def test_append_k_only():
    """A cache filled without queries."""
    Hkv, total = 2, 3
    k, v = _randn(_gen(93), total, Hkv, D), _randn(_gen(94), total, Hkv, D)
    kp, vp, table = pu.pools(1, [3], Hkv, 16, D, _gen(95), fill=0.0)
    tab, lens = _table(D, 8), pu.i32([3])
    gqa.gqa_packed_rope_append(None, 0, k, Hkv * D, v, Hkv * D, pu.i32([0, 3]), 1, total, 0, Hkv,
                               D, None, None, 0.0, tab, 8, None, None,
                               gqa.make_paged_kv(kp, vp, table, lens))
    assert pu.status() == 0
    assert torch.equal(vp[table[0, 0].long(), :, :3], v.transpose(0, 1))


@pytest.mark.parametrize("what,code", [("page", -1), ("negative", -1), ("table", -8), ("lens", -1),
                                       ("pages", -4)])
def test_append_bad_device_contents(what, code):
    """A page outside the pool, positions past the table, more new tokens than tokens, more
    tokens than pages: flagged, nothing written for that token, the other sequence served."""
    Hkv, t, s, page = 1, [2, 2], [20, 20], 16
    k = _randn(_gen(96), 4, D)
    kp, vp, table = pu.pools(2, s, Hkv, page, D, _gen(97), fill=0.0)
    good = table.clone()
    n_tab = 32
    tab = _table(D, n_tab)
    if what == "page":
        table[0, 1] = kp.shape[0]
    elif what == "negative":
        table[0, 1] = -1
    elif what == "table":
        n_tab = 19
    elif what == "lens":
        s = [1, 20]
    else:
        s = [33, 20]
    lens = pu.i32(s)
    gqa.gqa_packed_rope_append(None, 0, k, D, k, D, pu.i32(pu.cu_of(t)), 2, 4, 0, Hkv, D, None,
                               None, 0.0, tab, n_tab, None, None,
                               gqa.make_paged_kv(kp, vp, table, lens))
    assert pu.status() == code
    want = torch.zeros_like(vp)
    if what == "table":   # token 18 is inside the table, token 19 is not
        want[good[0, 1].long(), 0, 2] = k[0]
        want[good[1, 1].long(), 0, 2] = k[2]
    else:
        want[good[1, 1].long(), 0, 2] = k[2]
        want[good[1, 1].long(), 0, 3] = k[3]
    assert torch.equal(vp, want)


# ---- attention over the paged cache -----------------------------------------------------------

class Paged:
    """A batch over a paged cache whose unwritten rows hold NaN."""

    def __init__(self, t, s, Hq, Hkv, page, seed, max_q=None, max_kv=None, first=0, behind=0):
        gen = _gen(seed)
        self.t, self.s, self.Hq, self.Hkv, self.page = t, s, Hq, Hkv, page
        self.cu = pu.cu_of(t, first)
        self.total = self.cu[-1] + behind
        self.q = _randn(gen, self.total, Hq, D)
        self.q[:first] = math.nan
        self.q[self.cu[-1]:] = math.nan
        self.kp, self.vp, self.table = pu.pools(len(t), s, Hkv, page, D, gen)
        self.k, self.v = [], []
        for i, n in enumerate(s):
            self.k.append(_randn(gen, n, Hkv, D))
            self.v.append(_randn(gen, n, Hkv, D))
            pu.put(self.kp, self.table, i, self.k[-1])
            pu.put(self.vp, self.table, i, self.v[-1])
        self.max_q, self.max_kv = max_q or max(t), max_kv or max(s)
        self.cu_d, self.s_d = pu.i32(self.cu), pu.i32(s)
        self.cache = gqa.make_paged_kv(self.kp, self.vp, self.table, self.s_d)
        self.wsb = gqa.gqa_attn_paged_workspace_bytes(len(t), self.total, self.max_q, self.max_kv,
                                                      Hq, Hkv, D)
        # a workspace full of NaN: nothing may be read that this call did not write
        self.ws = torch.full((max(self.wsb, 16) // 4,), math.nan, device="cuda")
        self.o = torch.full((self.total, Hq * D + 8), -7.0, dtype=torch.bfloat16, device="cuda")
        self.L = torch.full((Hq, self.total), -7.0, device="cuda")

    def run(self, window=0, scale=D ** -0.5, stream=None):
        gqa.gqa_attn_paged(self.q, self.Hq * D, self.cache, self.cu_d, len(self.t), self.total,
                           self.max_q, self.max_kv, self.Hq, window, scale, self.o,
                           self.Hq * D + 8, self.L, self.ws, self.wsb, stream)

    def out(self):
        return self.o[:, :self.Hq * D].reshape(self.total, self.Hq, D)

    def check(self, window=0, scale=D ** -0.5, skip=()):
        o = self.out()
        assert (self.o[:, self.Hq * D:] == -7).all()
        for rows in (slice(0, self.cu[0]), slice(self.cu[-1], self.total)):
            assert (o[rows] == -7).all() and (self.L[:, rows] == -7).all()
        for i, n in enumerate(self.t):
            a, b = self.cu[i], self.cu[i + 1]
            if n == 0:
                continue
            if i in skip:
                assert (o[a:b] == -7).all() and (self.L[:, a:b] == -7).all()
                continue
            ro, rl, bo, bl = pu.attention64(self.q[a:b], self.k[i], self.v[i], window, scale)
            pu.check(o[a:b], ro, bo, f"o of sequence {i} ({n} of {self.s[i]})")
            pu.check(self.L[:, a:b], rl, bl, f"lse of sequence {i} ({n} of {self.s[i]})")


def _paged(t, s, Hq, Hkv, page, window, seed, **kw):
    p = Paged(t, s, Hq, Hkv, page, seed, **kw)
    p.run(window)
    st = pu.status()
    assert st == 0, gqa.STATUS_NAMES.get(st, st)
    p.check(window)
    return p


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (4, 4), (6, 2), (5, 1), (16, 1), (64, 1)])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("window", [0, 70])
def test_paged_decode(Hq, Hkv, page, window):
    _paged([1, 1, 0, 1, 1], [1, 137, 5, 300, 64], Hq, Hkv, page, window, 100 + Hq + page)


@pytest.mark.parametrize("t", [[2, 4, 1, 3], [8, 8, 7, 1], [5, 17, 2, 12]])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (6, 2), (2, 2)])
@pytest.mark.parametrize("window", [0, 1, 33])
def test_paged_drafts(t, Hq, Hkv, window):
    _paged(t, [2 + t[0], 200 + t[1], t[2], 515], Hq, Hkv, 16, window, 120 + Hq + window,
           behind=3)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (3, 3), (7, 1)])
@pytest.mark.parametrize("window", [0, 128, 300])
def test_paged_chunks(page, Hq, Hkv, window):
    """Whole prompts, chunks over a cache, single tokens and empty sequences in one batch."""
    _paged([200, 1, 0, 130, 64], [200, 500, 9, 900, 65], Hq, Hkv, page, window, 140 + Hq, first=3,
           behind=1)


@pytest.mark.parametrize("t", [1, 3, 40, 200])
@pytest.mark.parametrize("window", [0, 2048])
def test_paged_long(t, window):
    """One long sequence on few heads: its keys are split."""
    _paged([t], [9001], 8, 1, 64, window, 160 + t)


def test_paged_many_sequences():
    n = 150
    _paged([1] * n, [1 + (37 * i) % 400 for i in range(n)], 8, 2, 16, 0, 170)


def test_paged_many_ragged_drafts():
    n = 70
    _paged([i % 4 for i in range(n)], [3 + (53 * i) % 500 for i in range(n)], 8, 1, 32, 0, 171)


@pytest.mark.parametrize("t", [[1, 1, 1], [3, 1, 2], [150, 1, 20]])
def test_paged_loose_bounds(t):
    """max_q and max_kv far above the batch: the same results to the bound."""
    _paged(t, [300, 40, 129], 8, 2, 16, 0, 180, max_q=max(t) + 4, max_kv=20000)


@pytest.mark.parametrize("t", [[1, 1], [4, 2], [100, 1]])
def test_paged_bounds_exceeded(t):
    """A sequence above max_kv is skipped and flagged, the other one served."""
    p = Paged(t, [400, 150], 8, 2, 16, 190, max_kv=max(t[0], 200))
    p.run()
    assert pu.status() == -4
    p.check(skip=(0,))


@pytest.mark.parametrize("t", [[1, 1], [4, 2], [100, 1]])
def test_paged_more_queries_than_keys(t):
    p = Paged(t, [400, 150], 8, 2, 16, 191)
    p.s_d[0] = t[0] - 1
    p.run()
    assert pu.status() == -1
    p.check(skip=(0,))


@pytest.mark.parametrize("t", [[1, 1], [3, 1], [90, 1]])
@pytest.mark.parametrize("bad", [-1, None, 2 ** 31 - 1])
def test_paged_bad_page(t, bad):
    """A visible page outside the pool: flagged, read as zeros, the other sequence exact."""
    p = Paged(t, [300, 150], 8, 2, 16, 192)
    p.table[0, 4] = p.kp.shape[0] if bad is None else bad
    p.run()
    assert pu.status() == -1
    p.k[0][64:80] = 0
    p.v[0][64:80] = 0
    p.check()


@pytest.mark.parametrize("t", [[1, 1], [3, 2], [90, 1]])
def test_paged_pages_below_the_window_are_not_read(t):
    """Table entries of pages wholly below every window may be stale."""
    window, s = 100, [700, 333]
    p = Paged(t, s, 8, 2, 16, 193)
    for i in range(2):
        lo = s[i] - t[i] - window + 1
        p.table[i, :max(0, lo // 16)] = -5
    p.run(window)
    assert pu.status() == 0
    p.check(window)


@pytest.mark.parametrize("t", [1, 4, 70])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_paged_hidden_values_do_not_leak(t, window, bad):
    """A non-finite value at the last token and one in the middle: the rows that do not see
    them are those of the clean cache."""
    s, Hq, Hkv = 500, 8, 2
    p = Paged([t], [s], Hq, Hkv, 16, 194)
    p.run(window)
    clean = p.out().clone()
    L = p.L.clone()
    mid = s - t - 39
    for j in (mid, s - 1):
        p.vp[p.table[0, j // 16].long(), :, j % 16] = bad
    p.run(window)
    assert pu.status() == 0
    pos = torch.arange(s - t, s, device="cuda")
    sees = pos == s - 1
    sees |= (pos - mid < window) if window else torch.ones_like(sees)
    assert torch.equal(p.out()[~sees], clean[~sees])
    assert not torch.isfinite(p.out()[sees]).any()
    assert torch.equal(p.L, L)


def test_paged_shared_prefix_pages():
    """Two sequences whose first pages are the same ones."""
    p = Paged([1, 5], [100, 90], 8, 2, 16, 195)
    p.table[1, :4] = p.table[0, :4]
    p.k[1][:64], p.v[1][:64] = p.k[0][:64], p.v[0][:64]
    p.run()
    assert pu.status() == 0
    p.check()


@pytest.mark.parametrize("t,s", [([1] * 6, [3000, 10, 700, 1, 90, 2500]),
                                 ([2, 4, 1], [3000, 10, 700]), ([300, 1, 77], [3000, 10, 700])])
def test_paged_same_bits_every_run(t, s):
    p = Paged(t, s, 16, 2, 16, 196)
    p.run()
    a, l = p.o.clone(), p.L.clone()
    for _ in range(3):
        p.ws.fill_(1e30)
        p.run()
        assert torch.equal(p.o, a) and torch.equal(p.L, l)
    assert pu.status() == 0


@pytest.mark.parametrize("t,s", [([1, 1, 1], [300, 40, 1]), ([3, 1, 2], [64, 300, 40]),
                                 ([140, 1, 0], [200, 300, 40])])
def test_paged_capture_follows_the_lengths(t, s):
    """A captured call replayed after the lengths, the pages and the queries changed."""
    p = Paged(t, s, 8, 2, 16, 197, max_kv=512)
    p.run()                                   # loads the kernels before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        p.run()
    torch.cuda.current_stream().wait_stream(side)
    # the same buffers, new contents: longer sequences in as many pages
    p2 = Paged(t, [min(n + 5, (n + 15) // 16 * 16) for n in s], 8, 2, 16, 197, max_kv=512)
    assert p2.kp.shape == p.kp.shape and p2.table.shape == p.table.shape
    for a, b in ((p.q, p2.q), (p.kp, p2.kp), (p.vp, p2.vp), (p.table, p2.table),
                 (p.s_d, p2.s_d)):
        a.copy_(b)
    p.k, p.v, p.s = p2.k, p2.v, p2.s
    p.o.fill_(-7)
    p.L.fill_(-7)
    p.ws.fill_(math.nan)
    g.replay()
    torch.cuda.synchronize()
    assert pu.status() == 0
    p.check()


def test_paged_two_calls_at_once():
    """Two calls on two streams with a workspace each."""
    ps = [Paged([1] * 4, [4000, 30, 1000, 512], 8, 2, 16, 199 + i) for i in range(2)]
    ss = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s in zip(ps, ss):
            p.run(stream=s)
    torch.cuda.synchronize()
    assert pu.status() == 0
    for p in ps:
        p.check()


@pytest.mark.parametrize("t", [1, 2, 40])
def test_paged_pool_beyond_32_bit_offsets(t):
    """Pages whose elements lie beyond 2^31 of the pool's start."""
    Hq, Hkv, page, s = 16, 8, 16, 100
    pages = 2 ** 31 // (Hkv * page * D) + 64
    p = Paged([t], [s], Hq, Hkv, page, 203)
    kp = torch.zeros(pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    n = p.kp.shape[0]
    kp[-n:], vp[-n:] = p.kp, p.vp
    p.table += pages - n
    p.kp, p.vp = kp, vp
    p.table.clamp_(max=pages - 1)
    p.cache = gqa.make_paged_kv(kp, vp, p.table, p.s_d)
    p.run()
    assert pu.status() == 0
    p.check()


# ---- a run of them together -----------------------------------------------------------------------

@pytest.mark.parametrize("window", [0, 48])
def test_steps_over_a_paged_cache_equal_whole_prompts(window):
    """Two sequences grow in a prompt chunk, further chunks, a draft and single tokens, append
    then attention each time; every output equals one packed pass over the whole sequences."""
    Hq, Hkv, page, N = 8, 2, 16, [230, 150]
    gen = _gen(210)
    eps = 1e-6
    xs = [_randn(gen, n, (Hq + 2 * Hkv) * D) for n in N]
    gq, gk = (1 + 0.1 * torch.randn(D, generator=gen)).cuda(), torch.ones(D, device="cuda")
    tab = _table(D, 256)
    row = (Hq + 2 * Hkv) * D
    steps = [(100, 0), (100, 64), (3, 5), (1, 1), (1, 0), (0, 2), (25, 78)]
    kp, vp, table = pu.pools(2, N, Hkv, page, D, gen)
    got = [[], []]
    done = [0, 0]
    for ts in steps:
        x = torch.cat([xs[i][done[i]:done[i] + ts[i]] for i in range(2)])
        done = [a + b for a, b in zip(done, ts)]
        total, cu, lens = x.shape[0], pu.i32(pu.cu_of(ts)), pu.i32(done)
        q, k, v = x.split([Hq * D, Hkv * D, Hkv * D], 1)
        qr = torch.empty(total, Hq, D, dtype=torch.bfloat16, device="cuda")
        o = torch.empty_like(qr)
        cache = gqa.make_paged_kv(kp, vp, table, lens)
        gqa.gqa_packed_rope_append(q, row, k, row, v, row, cu, 2, total, Hq, Hkv, D, gq, gk, eps,
                                   tab, 256, qr, None, cache)
        a = (2, total, max(ts), max(done), Hq, Hkv, D)
        wsb = gqa.gqa_attn_paged_workspace_bytes(*a)
        ws = torch.full((max(wsb, 16) // 4,), math.nan, device="cuda")
        gqa.gqa_attn_paged(qr, Hq * D, cache, cu, 2, total, max(ts), max(done), Hq, window,
                           D ** -0.5, o, Hq * D, None, ws, wsb)
        assert pu.status() == 0
        got[0].append(o[:ts[0]])
        got[1].append(o[ts[0]:])
    assert done == N
    # the same tokens in one packed pass without a cache
    x = torch.cat(xs)
    total, cu = sum(N), pu.i32(pu.cu_of(N))
    q, k, v = x.split([Hq * D, Hkv * D, Hkv * D], 1)
    qr = torch.empty(total, Hq, D, dtype=torch.bfloat16, device="cuda")
    kr = torch.empty(total, Hkv, D, dtype=torch.bfloat16, device="cuda")
    o = torch.empty_like(qr)
    gqa.gqa_packed_rope_append(q, row, k, row, None, 0, cu, 2, total, Hq, Hkv, D, gq, gk, eps, tab,
                               256, qr, kr, None)
    gqa.gqa_attn_packed(qr, Hq * D, kr, Hkv * D, v, row, o, Hq * D, None, cu, 2, total, Hq, Hkv, D,
                        window, D ** -0.5)
    assert pu.status() == 0
    at = 0
    for i, n in enumerate(N):
        vi = v[at:at + n].reshape(n, Hkv, D)
        ro, _, bo, _ = pu.attention64(qr[at:at + n], kr[at:at + n], vi, window, D ** -0.5)
        pu.check(torch.cat(got[i]), ro, bo, f"steps of sequence {i}")
        pu.check(o[at:at + n], ro, bo, f"packed pass of sequence {i}")
        at += n
