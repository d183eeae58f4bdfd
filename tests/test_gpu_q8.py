"""The 8-bit paged cache on the GPU: gqa_packed_rope_append_q8, gqa_attn_paged_q8 and
gqa_paged_read_q8 against plain 64-bit forms, at the sizes, masks, strides and contents where
they can go wrong."""
import math

import pytest
import torch

import global_causal_gqa_gb300 as gqa
import gpu_utils as gu
import packed_utils as pu
import q8_utils as q8
from test_gpu_packed import D, _gen, _randn, _table

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


# ---- the append ---------------------------------------------------------------------------------

def _append(d, page, norm, Hq, Hkv, t, past, seed, edit=None, amp=1.25, k_out=True, q=True):
    """One call over pools full of NaN; returns what a test compares."""
    gen = _gen(seed)
    eps, total = 1e-6, sum(t) + 2
    cu = pu.cu_of(t, 1)
    s = [a + b for a, b in zip(t, past)]
    qkv = _randn(gen, total, (Hq + 2 * Hkv) * d + 8)     # rows wider than their three parts
    row = qkv.shape[1]
    xq, xk, xv, _ = qkv.split([Hq * d, Hkv * d, Hkv * d, 8], 1)
    if edit:
        edit(xk, xv)
    gq = (1 + 0.1 * torch.randn(d, generator=gen)).cuda() if norm else None
    gk = (1 + 0.1 * torch.randn(d, generator=gen)).cuda() if norm else None
    kq, vq, sc, table = q8.pools(len(t), s, Hkv, page, d, gen)
    lens, tab = pu.i32(s), _table(d, max(s), amp=amp)
    qo = torch.full((total, Hq, d), -7.0, dtype=torch.bfloat16, device="cuda") if q else None
    ko = torch.full((total, Hkv, d), -7.0, dtype=torch.bfloat16, device="cuda") if k_out else None
    gqa.gqa_packed_rope_append_q8(xq if q else None, row, xk, row, xv, row, pu.i32(cu), len(t),
                                  total, Hq if q else 0, Hkv, d, gq if q else None, gk, eps, tab,
                                  max(s), qo, ko, q8.cache_of(kq, vq, sc, table, lens))
    st = pu.status()
    assert st == 0, gqa.STATUS_NAMES.get(st, st)
    pos = torch.tensor([p + i for n, p in zip(t, past) for i in range(n)], device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(t)), torch.tensor(t)).cuda()
    pg, slot = table.long()[seq, pos // page], pos % page
    r = slice(cu[0], cu[-1])
    return dict(q=xq.reshape(total, Hq, d)[r], k=xk.reshape(total, Hkv, d)[r],
                v=xv.reshape(total, Hkv, d)[r], gq=gq, gk=gk, eps=eps, amp=amp, pos=pos, qo=qo,
                ko=ko, r=r, kq=kq, vq=vq, sc=sc, pg=pg, slot=slot)


def _rope_bound(x, d):
    """fp32 roundings of the table, the norm's sum of d squares and the products, relative to a
    pair's length; below 2^-126 fp32's step is 2^-149, and half a step is lost by each of two
    products and their sum."""
    h = x.abs()
    pair = torch.cat([h[..., :d // 2] + h[..., d // 2:]] * 2, -1)
    return (16 + d) * pu.FP32 * pair * 1.5 + 3 * 2.0 ** -150


BF16_SUB = 2.0 ** -134     # half of bf16's step below 2^-126, 2^-133


def _check_append(x, d):
    if x["qo"] is not None:
        ref = pu.rope64(x["q"], x["pos"], 1e4, x["gq"], x["eps"], x["amp"])
        pu.check(x["qo"][x["r"]], ref, pu.BF16 * ref.abs() + _rope_bound(ref, d), "q_out")
        assert (x["qo"][:x["r"].start] == -7).all() and (x["qo"][x["r"].stop:] == -7).all()
    ref = pu.rope64(x["k"], x["pos"], 1e4, x["gk"], x["eps"], x["amp"])
    off = _rope_bound(ref, d)
    if x["ko"] is not None:
        pu.check(x["ko"][x["r"]], ref, pu.BF16 * ref.abs() + off + BF16_SUB, "k_out")
    # values: the same bits as the plain form's
    data, byte = q8.quantise(x["v"])
    assert torch.equal(x["sc"][x["pg"], :, x["slot"], 1], byte)
    assert torch.equal(x["vq"][x["pg"], :, x["slot"]], data)
    # keys: the byte of a largest element within its error; each number within half a step
    data, byte = x["kq"][x["pg"], :, x["slot"]], x["sc"][x["pg"], :, x["slot"], 0]
    most, far = ref.abs().amax(-1), off.amax(-1)
    assert ((byte >= q8.scale_bytes((most - far).clamp_min(0))) &
            (byte <= q8.scale_bytes(most + far))).all()
    step = q8.power(byte)[..., None]
    pu.check(q8.values(data, byte), ref, off + torch.maximum(q8.E4M3 * (ref.abs() + off),
                                                             q8.TINY * step) +
             (ref.abs() - 448 * step).clamp_min(0), "keys")
    # nothing else was written
    for pool, fill in ((x["kq"], 0x7f), (x["vq"], 0x7f), (x["sc"], 255)):
        rest = pool.clone()
        rest[x["pg"], :, x["slot"]] = fill
        assert (rest == fill).all()


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("Hq,Hkv,t,past", [(8, 2, [1], [137]), (5, 5, [3, 0, 40], [0, 7, 16]),
                                           (64, 8, [1] * 9, [0, 15, 16, 17, 31, 5, 6, 100, 127]),
                                           (3, 1, [70, 259], [1, 0]),
                                           (4, 3, [609, 1, 700], [3, 0, 33])])
def test_append(d, page, norm, Hq, Hkv, t, past):
    _check_append(_append(d, page, norm, Hq, Hkv, t, past, 81 + d + Hq), d)


@pytest.mark.parametrize("Hq,Hkv,d", [(64, 8, 128), (40, 8, 512), (3, 7, 64)])
def test_append_many_tokens(Hq, Hkv, d):
    """The streamed form, whose units are runs of a token's vectors where these are long."""
    _check_append(_append(d, 32, True, Hq, Hkv, [1000, 0, 333, 5], [0, 9, 100, 31], 91 + d), d)


@pytest.mark.parametrize("n", [3, 700])
def test_append_without_queries_or_k_out(n):
    _check_append(_append(D, 16, False, 1, 2, [n, 2], [5, 0], 95, k_out=False, q=False), D)


@pytest.mark.parametrize("n", [5, 700])
@pytest.mark.parametrize("d", [64, 128, 512])
def test_append_extremes(n, d):
    """Zero vectors, the largest and smallest magnitudes, a single element, borders of the power
    of two (448 * 2^e exactly, and the next bf16 number)."""
    big = 3.3895313892515355e38
    rows = [0.0, big, -big, 1e-38, 2.0 ** -133, 448.0, 450.0, 448 * 2.0 ** 60, 2.0 ** -119, 7.0,
            224.0, 226.0]

    def edit(k, v):
        for i, x in enumerate(rows):
            if i < n:
                v[1 + i] = x
                k[1 + i] = 0 if abs(x) > 1e37 else x
        v[1].view(-1)[3] = -5e-39
        v[n] = 0
        v[n, 1] = -3.0
    _check_append(_append(d, 16, False, 2, 1, [n], [11], 97, edit=edit, amp=1.0), d)


@pytest.mark.parametrize("n", [6, 700])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_append_nonfinite(n, bad):
    """A vector with a non-finite element is stored as NaN whole; the others as without it."""
    def edit(k, v):
        k[3, 5] = bad
        v[2, 127] = bad
        v[n, 128 + 64] = bad
    clean = _append(D, 16, True, 2, 2, [n], [40], 99)
    dirty = _append(D, 16, True, 2, 2, [n], [40], 99, edit=edit)
    want_k, want_v, want_s = clean["kq"].clone(), clean["vq"].clone(), clean["sc"].clone()
    for pool, which, t, h in ((want_k, 0, 2, 0), (want_v, 1, 1, 0), (want_v, 1, n - 1, 1)):
        pg, slot = clean["pg"][t], clean["slot"][t]
        pool[pg, h, slot] = 0
        want_s[pg, h, slot, which] = 255
    assert torch.equal(dirty["kq"], want_k) and torch.equal(dirty["vq"], want_v)
    assert torch.equal(dirty["sc"], want_s)


@pytest.mark.parametrize("what,code", [("page", -1), ("negative", -1), ("table", -8), ("lens", -1),
                                       ("pages", -4)])
@pytest.mark.parametrize("n", [2, 650])
def test_append_bad_device_contents(what, code, n):
    """Flagged, nothing written for those tokens, the other sequence served."""
    t, s = [2, n], [20, n + 18]
    k = _randn(_gen(96), n + 2, D)
    kq, vq, sc, table = q8.pools(2, s, 1, 16, D, _gen(97))
    good = table.clone()
    n_tab = n + 40
    if what == "page":
        table[0, 1] = kq.shape[0]
    elif what == "negative":
        table[0, 1] = -1
    elif what == "table":
        n_tab = n + 17
    elif what == "lens":
        s = [1, s[1]]
    else:
        s = [16 * table.shape[1] + 1, s[1]]
    tab = _table(D, n + 40)
    gqa.gqa_packed_rope_append_q8(None, 0, k, D, k, D, pu.i32(pu.cu_of(t)), 2, n + 2, 0, 1, D,
                                  None, None, 0.0, tab, n_tab, None, None,
                                  q8.cache_of(kq, vq, sc, table, pu.i32(s)))
    assert pu.status() == code
    want = torch.full_like(vq, 0x7f)
    data, _ = q8.quantise(k)
    for i, (a, first, m) in enumerate(((0, 18, 2), (2, 18, n))):
        if i == 0 and what != "table":
            continue
        j = torch.arange(first, first + m, device="cuda")
        j = j[j < n_tab]
        pg, slot = q8.places(good, i, 16, j)
        want[pg, 0, slot] = data[a:a + len(j)]
    assert torch.equal(vq, want)


# ---- reading back ---------------------------------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("page", [16, 64])
def test_read_every_number(d, page):
    """Every pair of an e4m3 number and a scale byte, against the plain product rounded to bf16."""
    n = 256 * 256 // d
    x = torch.arange(256 * 256, device="cuda")
    data = (x % 256).to(torch.uint8).reshape(n, 1, d)
    byte = (x // 256)[::d].to(torch.uint8).reshape(n, 1)
    kq, vq, sc, table = q8.pools(1, [n], 1, page, d, _gen(3))
    j = torch.arange(n, device="cuda")
    pg, slot = q8.places(table, 0, page, j)
    kq[pg, :, slot], vq[pg, :, slot] = data, data.flip(0)
    sc[pg, :, slot, 0], sc[pg, :, slot, 1] = byte, byte.flip(0)
    ko = torch.empty(n, 1, d, dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)
    gqa.gqa_paged_read_q8(q8.cache_of(kq, vq, sc, table, pu.i32([n])), pu.i32([0, n]), 1, n, ko, d,
                          vo, d)
    assert pu.status() == 0
    want = q8.values(data, byte).float().to(torch.bfloat16)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(ko), nan)
    assert torch.equal(ko[~nan], want[~nan])
    assert torch.equal(torch.isnan(vo), nan.flip(0))
    assert torch.equal(vo[~nan.flip(0)], want.flip(0)[~nan.flip(0)])


def _random_cache(s, Hkv, page, d, seed):
    gen = _gen(seed)
    kq, vq, sc, table = q8.pools(len(s), s, Hkv, page, d, gen)
    rows = []
    for i, n in enumerate(s):
        x = [q8.quantise(_randn(gen, n, Hkv, d)) for _ in range(2)]
        pg, slot = q8.places(table, i, page, torch.arange(n, device="cuda"))
        kq[pg, :, slot], vq[pg, :, slot] = x[0][0], x[1][0]
        sc[pg, :, slot, 0], sc[pg, :, slot, 1] = x[0][1], x[1][1]
        rows.append(x)
    return kq, vq, sc, table, rows


@pytest.mark.parametrize("d,Hkv", [(64, 1), (128, 2), (128, 7), (256, 3), (512, 2)])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("t,s", [([1], [1]), ([17], [120]), ([3, 0, 40, 200], [3, 5, 90, 333]),
                                 ([0] * 20 + [1, 2] * 30, [4] * 80)])
def test_read(d, Hkv, page, t, s):
    """The newest tokens of each sequence, into rows with a stride, rows of no sequence left."""
    kq, vq, sc, table, rows = _random_cache(s, Hkv, page, d, 7 + d)
    cu = pu.cu_of(t, 2)
    total = cu[-1] + 3
    out = torch.full((2, total, Hkv * d + 8), -7.0, dtype=torch.bfloat16, device="cuda")
    lens = pu.i32(s)
    cache = q8.cache_of(kq, vq, sc, table, lens)
    gqa.gqa_paged_read_q8(cache, pu.i32(cu), len(t), total, out[0], Hkv * d + 8, out[1],
                          Hkv * d + 8)
    assert pu.status() == 0
    want = torch.full_like(out, -7.0)
    for i, (a, b) in enumerate(zip(t, s)):
        for w in range(2):
            x = q8.values(*rows[i][w])[b - a:].to(torch.bfloat16)
            want[w, cu[i]:cu[i + 1], :Hkv * d] = x.reshape(a, Hkv * d)
    assert torch.equal(out, want)
    only = torch.full_like(out[0], -7.0)
    gqa.gqa_paged_read_q8(cache, pu.i32(cu), len(t), total, None, 0, only, Hkv * d + 8)
    assert torch.equal(only, want[1])
    only.fill_(-7)
    gqa.gqa_paged_read_q8(cache, pu.i32(cu), len(t), total, only, Hkv * d + 8, None, 0)
    assert torch.equal(only, want[0])


@pytest.mark.parametrize("what,code", [("page", -1), ("lens", -1), ("pages", -4), ("cu", -1)])
def test_read_bad_device_contents(what, code):
    """A page outside the pool reads as zeros; a sequence whose numbers do not fit is left."""
    t, s = [30, 5], [40, 9]
    kq, vq, sc, table, rows = _random_cache(s, 2, 16, D, 11)
    cu = pu.cu_of(t)
    if what == "page":
        table[0, 1] = -3
    elif what == "lens":
        s = [29, 9]
    elif what == "pages":
        s = [16 * table.shape[1] + 1, 9]
    else:
        cu = [0, -4, 5]
        cu = [-1, 30, 35]
    out = torch.full((2, 35, 2, D), -7.0, dtype=torch.bfloat16, device="cuda")
    lens = pu.i32(s)
    gqa.gqa_paged_read_q8(q8.cache_of(kq, vq, sc, table, lens), pu.i32(cu), 2, 35, out[0], 2 * D,
                          out[1], 2 * D)
    assert pu.status() == code
    for w in range(2):
        assert torch.equal(out[w, 30:], q8.values(*rows[1][w])[4:].to(torch.bfloat16))
        if what == "page":
            want = q8.values(*rows[0][w])[10:].to(torch.bfloat16)
            want[6:22] = 0
            assert torch.equal(out[w, :30], want)
        else:
            assert (out[w, :30] == -7).all()


# ---- attention ------------------------------------------------------------------------------------

class PagedQ8:
    """A batch over an 8-bit cache whose unwritten numbers and bytes are NaN."""

    def __init__(self, t, s, Hq, Hkv, page, seed, max_q=None, max_kv=None, first=0, behind=0,
                 spread=0):
        gen = _gen(seed)
        self.t, self.s, self.Hq, self.Hkv, self.page = t, s, Hq, Hkv, page
        self.cu = pu.cu_of(t, first)
        self.total = self.cu[-1] + behind
        self.q = _randn(gen, self.total, Hq, D)
        self.q[:first] = math.nan
        self.q[self.cu[-1]:] = math.nan
        self.kq, self.vq, self.sc, self.table = q8.pools(len(t), s, Hkv, page, D, gen)
        n, x = sum(s), []
        for _ in range(2):
            y = _randn(gen, n, Hkv, D)
            # powers of two of their own for every vector, over `spread` binades
            up = torch.randint(0, spread + 1, (n, Hkv, 1), generator=gen).cuda() - spread
            x += list(q8.quantise(y.double() * torch.exp2(up.double())))
        # of each sequence: key numbers, key bytes, value numbers, value bytes
        self.rows = [list(parts) for parts in zip(*(y.split(s) for y in x))]
        seq = torch.repeat_interleave(torch.arange(len(s)), torch.tensor(s)).cuda()
        at = torch.cat([torch.arange(n) for n in s]).cuda()
        self.write(self.table.long()[seq, at // page], at % page, x)
        self.max_q, self.max_kv = max_q or max(t), max_kv or max(s)
        self.cu_d, self.s_d = pu.i32(self.cu), pu.i32(s)
        self.cache = q8.cache_of(self.kq, self.vq, self.sc, self.table, self.s_d)
        self.wsb = gqa.gqa_attn_paged_q8_workspace_bytes(len(t), self.total, self.max_q,
                                                         self.max_kv, Hq, Hkv, D)
        # a workspace full of NaN: nothing may be read that this call did not write
        self.ws = torch.full((max(self.wsb, 16) // 4 + 1,), math.nan, device="cuda")
        self.o = torch.full((self.total, Hq * D + 8), -7.0, dtype=torch.bfloat16, device="cuda")
        self.L = torch.full((Hq, self.total), -7.0, device="cuda")

    def write(self, pg, slot, x):
        self.kq[pg, :, slot], self.vq[pg, :, slot] = x[0], x[2]
        self.sc[pg, :, slot, 0], self.sc[pg, :, slot, 1] = x[1], x[3]

    def put(self, i):
        n = self.rows[i][0].shape[0]
        self.write(*q8.places(self.table, i, self.page, torch.arange(n, device="cuda")), self.rows[i])

    def run(self, window=0, scale=D ** -0.5, stream=None):
        gqa.gqa_attn_paged_q8(self.q, self.Hq * D, self.cache, self.cu_d, len(self.t), self.total,
                              self.max_q, self.max_kv, self.Hq, window, scale, self.o,
                              self.Hq * D + 8, self.L, self.ws, self.wsb, stream)

    def out(self):
        return self.o[:, :self.Hq * D].reshape(self.total, self.Hq, D)

    def check(self, window=0, scale=D ** -0.5, skip=(), only=None):
        """only: the sequences that are looked at (None: all); those of `skip` have to be as they
        were."""
        o = self.out()
        assert (self.o[:, self.Hq * D:] == -7).all()
        for rows in (slice(0, self.cu[0]), slice(self.cu[-1], self.total)):
            assert (o[rows] == -7).all() and (self.L[:, rows] == -7).all()
        for i, n in enumerate(self.t):
            a, b = self.cu[i], self.cu[i + 1]
            if n == 0 or (only is not None and i not in only):
                continue
            if i in skip:
                assert (o[a:b] == -7).all() and (self.L[:, a:b] == -7).all()
                continue
            ro, rl, bo, bl = q8.attention64(self.q[a:b], *self.rows[i], window, scale)
            pu.check(o[a:b], ro, bo, f"o of sequence {i} ({n} of {self.s[i]})")
            pu.check(self.L[:, a:b], rl, bl, f"lse of sequence {i} ({n} of {self.s[i]})")


def _paged(t, s, Hq, Hkv, page, window, seed, scale=D ** -0.5, only=None, **kw):
    p = PagedQ8(t, s, Hq, Hkv, page, seed, **kw)
    p.run(window, scale)
    st = pu.status()
    assert st == 0, gqa.STATUS_NAMES.get(st, st)
    p.check(window, scale, only=only)
    return p


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (4, 4), (6, 2), (5, 1), (16, 1), (64, 1)])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("window", [0, 70])
def test_decode(Hq, Hkv, page, window):
    _paged([1, 1, 0, 1, 1], [1, 137, 5, 300, 64], Hq, Hkv, page, window, 100 + Hq + page)


@pytest.mark.parametrize("t", [[2, 4, 1, 3], [8, 8, 7, 1], [5, 17, 2, 12]])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (6, 2), (2, 2)])
@pytest.mark.parametrize("window", [0, 1, 33])
def test_drafts(t, Hq, Hkv, window):
    _paged(t, [2 + t[0], 200 + t[1], t[2], 515], Hq, Hkv, 16, window, 120 + Hq + window, behind=3)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (3, 3), (7, 1)])
@pytest.mark.parametrize("window", [0, 128, 300])
def test_chunks(page, Hq, Hkv, window):
    """Whole prompts, chunks over a cache, single tokens and empty sequences in one batch."""
    _paged([200, 1, 0, 130, 64], [200, 500, 9, 900, 65], Hq, Hkv, page, window, 140 + Hq, first=3,
           behind=1)


@pytest.mark.parametrize("t", [1, 2, 3, 6, 40, 200])
@pytest.mark.parametrize("window", [0, 2048])
@pytest.mark.parametrize("page", [16, 64])
def test_long(t, window, page):
    """One long sequence on few heads: its keys are split."""
    _paged([t], [9001], 8, 1, page, window, 160 + t)


@pytest.mark.parametrize("t", [1, 2, 5, 70])
def test_spread_scales(t):
    """Powers of two that differ by up to 2^20 between neighbouring keys and values."""
    _paged([t, t], [700, 90], 8, 2, 16, 0, 165 + t, spread=20)


@pytest.mark.parametrize("t", [1, 2, 5])
@pytest.mark.parametrize("far", [-100, 100])
def test_far_value_scales(t, far):
    """A value 2^100 times the others at a key of no weight, or all but one value 2^100 times
    smaller: neither range of numbers swallows the other's part."""
    p = PagedQ8([t], [900], 8, 1, 16, 166)
    kd, kb, vd, vb = p.rows[0]
    u = p.q[0, 0].double()
    p.q[:] = p.q[0, 0]                     # every row the same query
    # one key far below all others in score (-300), its value 2^far times the others
    y, b = q8.quantise((-300 * u * D ** 0.5 / u.dot(u))[None, None])
    for at in (5, 640):
        kd[at], kb[at] = y[0], b[0]
        vb[at] = (vb[at].int() + far).clamp(1, 246).to(torch.uint8)
    p.put(0)
    p.run()
    assert pu.status() == 0
    p.check()


@pytest.mark.parametrize("t", [1, 2, 5, 100])
@pytest.mark.parametrize("scale", [1e-3, 4.0])
def test_scales(t, scale):
    """Flat weights, and weights of which a few carry all."""
    _paged([t, 1], [400, 31], 8, 2, 16, 0, 167, scale=scale)


@pytest.mark.parametrize("t", [1, 3, 100])
def test_rising_scores(t):
    """The row maximum grows with every key: the running rescale is taken each time."""
    p = PagedQ8([t], [1500], 8, 1, 16, 168)
    p.q[:] = p.q[0, 0]
    u = p.q[0, 0].double()
    x = torch.linspace(-60, 60, 1500, device="cuda", dtype=torch.float64)[:, None, None]
    p.rows[0][0], p.rows[0][1] = q8.quantise(x * (u * D ** 0.5 / u.dot(u)))
    p.put(0)
    p.run()
    assert pu.status() == 0
    p.check()


@pytest.mark.parametrize("t", [1, 2, 40])
@pytest.mark.parametrize("mag", [2.0 ** -60, 2.0 ** 40])
def test_query_magnitudes(t, mag):
    """Queries far outside f16's range, with keys the other way."""
    p = PagedQ8([t], [300], 8, 2, 32, 169)
    p.q.mul_(mag)
    e = int(math.log2(mag))
    p.rows[0][1].copy_((p.rows[0][1].int() - e).to(torch.uint8))
    p.q[:, 1, 3:] = 0                      # a row of few elements, one of none
    p.q[:, 2] = 0
    p.put(0)
    p.run()
    assert pu.status() == 0
    p.check()


def test_many_sequences():
    n = 150
    _paged([1] * n, [1 + (37 * i) % 400 for i in range(n)], 8, 2, 16, 0, 170)
    _paged([1] * n, [1 + (37 * i) % 900 for i in range(n)], 8, 2, 16, 0, 170)


@pytest.mark.parametrize("G", [4, 8])
def test_many_ragged_drafts(G):
    n = 70
    _paged([i % 4 for i in range(n)], [3 + (53 * i) % 700 for i in range(n)], G, 1, 32, 0, 171)
    _paged([i % 7 for i in range(n)], [7 + (53 * i) % 700 for i in range(n)], G, 1, 32, 0, 172)


@pytest.mark.parametrize("t", [[1, 1, 1], [3, 1, 2], [150, 1, 20]])
def test_loose_bounds(t):
    """max_q and max_kv far above the batch: the same results to the bound."""
    _paged(t, [300, 40, 129], 8, 2, 16, 0, 180, max_q=max(t) + 4, max_kv=20000)


@pytest.mark.parametrize("t", [[1, 1], [4, 2], [100, 1]])
def test_bounds_exceeded(t):
    """A sequence above max_kv is skipped and flagged, the other one served."""
    p = PagedQ8(t, [400, 150], 8, 2, 16, 190, max_kv=max(t[0], 200))
    p.run()
    assert pu.status() == -4
    p.check(skip=(0,))


@pytest.mark.parametrize("t", [[1, 1], [4, 2], [100, 1]])
def test_more_keys_than_pages(t):
    """A sequence longer than its row of the page table, but not than max_kv."""
    p = PagedQ8(t, [400, 150], 8, 2, 16, 189, max_kv=1000)
    p.s_d[0] = 401
    p.run()
    assert pu.status() == -4
    p.check(skip=(0,))


@pytest.mark.parametrize("t", [[1, 1], [4, 2], [100, 1]])
def test_more_queries_than_keys(t):
    p = PagedQ8(t, [400, 150], 8, 2, 16, 191)
    p.s_d[0] = t[0] - 1
    p.run()
    assert pu.status() == -1
    p.check(skip=(0,))


@pytest.mark.parametrize("t", [[1, 1], [3, 1], [90, 1]])
@pytest.mark.parametrize("bad", [-1, None, 2 ** 31 - 1])
def test_bad_page(t, bad):
    """A visible page outside the pool: flagged, read as zeros, the other sequence exact."""
    p = PagedQ8(t, [300, 150], 8, 2, 16, 192)
    p.table[0, 4] = p.kq.shape[0] if bad is None else bad
    p.run()
    assert pu.status() == -1
    for x in p.rows[0][0], p.rows[0][2]:
        x[64:80] = 0
    p.check()


@pytest.mark.parametrize("t", [[1, 1], [3, 2], [90, 1]])
def test_pages_below_the_window_are_not_read(t):
    """Table entries of pages wholly below every window may be stale."""
    window, s = 100, [700, 333]
    p = PagedQ8(t, s, 8, 2, 16, 193)
    for i in range(2):
        lo = s[i] - t[i] - window + 1
        p.table[i, :max(0, lo // 16)] = -5
    p.run(window)
    assert pu.status() == 0
    p.check(window)


@pytest.mark.parametrize("t", [1, 3, 4, 70])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("how", ["byte", "number"])
def test_hidden_values_do_not_leak(t, window, how):
    """A NaN value at the last token and one in the middle, by its byte or by a number of it: the
    rows that do not see them are those of the clean cache."""
    s, Hq, Hkv = 500, 8, 2
    p = PagedQ8([t], [s], Hq, Hkv, 16, 194)
    p.run(window)
    clean, L = p.out().clone(), p.L.clone()
    mid = s - t - 39
    for j in (mid, s - 1):
        if how == "byte":
            p.sc[p.table[0, j // 16].long(), :, j % 16, 1] = 255
        else:
            p.vq[p.table[0, j // 16].long(), :, j % 16, 77] = 0xff
    p.run(window)
    assert pu.status() == 0
    pos = torch.arange(s - t, s, device="cuda")
    sees = pos == s - 1
    sees |= (pos - mid < window) if window else torch.ones_like(sees)
    want = clean.clone()
    if how == "byte":
        want[sees] = math.nan
    else:
        want[sees, :, 77] = math.nan
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(p.out()), nan)
    assert torch.equal(p.out()[~nan], want[~nan])
    assert torch.equal(p.L, L)


@pytest.mark.parametrize("t", [1, 3, 70])
@pytest.mark.parametrize("how", ["byte", "number"])
def test_nan_keys(t, how):
    """A NaN key: NaN for the rows that see it, nothing for the others."""
    s = 300
    p = PagedQ8([t], [s], 8, 2, 32, 197)
    p.run()
    clean, L = p.out().clone(), p.L.clone()
    j = s - 1
    if how == "byte":
        p.sc[p.table[0, j // 32].long(), :, j % 32, 0] = 255
    else:
        p.kq[p.table[0, j // 32].long(), :, j % 32, 9] = 0x7f
    p.run()
    assert pu.status() == 0
    assert torch.equal(p.out()[:t - 1], clean[:t - 1]) and torch.equal(p.L[:, :t - 1], L[:, :t - 1])
    assert torch.isnan(p.out()[t - 1]).all() and torch.isnan(p.L[:, t - 1]).all()


@pytest.mark.parametrize("t", [1, 3, 70])
def test_nonfinite_queries(t):
    """A query row with a NaN: that row alone."""
    p = PagedQ8([t], [300], 8, 2, 32, 198)
    p.run()
    clean = p.out().clone()
    p.q[0, 3, 5] = math.nan
    p.run()
    assert pu.status() == 0
    want = clean.clone()
    want[0, 3] = math.nan
    assert torch.equal(torch.isnan(p.out()), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(p.out()[keep], clean[keep])


def test_shared_prefix_pages():
    """Two sequences whose first pages are the same ones."""
    p = PagedQ8([1, 5], [100, 90], 8, 2, 16, 195)
    p.table[1, :4] = p.table[0, :4]
    for x, y in zip(p.rows[1], p.rows[0]):
        x[:64] = y[:64]
    p.run()
    assert pu.status() == 0
    p.check()


@pytest.mark.parametrize("t,s", [([1] * 6, [3000, 10, 700, 1, 90, 2500]),
                                 ([2, 4, 1], [3000, 10, 700]), ([300, 1, 77], [3000, 10, 700])])
def test_same_bits_every_run(t, s):
    p = PagedQ8(t, s, 16, 2, 16, 196)
    p.run()
    a, l = p.o.clone(), p.L.clone()
    for _ in range(3):
        p.ws.fill_(1e30)
        p.run()
        assert torch.equal(p.o, a) and torch.equal(p.L, l)
    assert pu.status() == 0


@pytest.mark.parametrize("t,s", [([1, 1, 1], [300, 40, 1]), ([3, 1, 2], [64, 300, 40]),
                                 ([140, 1, 0], [200, 300, 40])])
def test_capture_follows_the_lengths(t, s):
    """A captured call replayed after the lengths, the pages and the queries changed."""
    p = PagedQ8(t, s, 8, 2, 16, 197, max_kv=600)
    p.run()                                   # loads the kernels before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        p.run()
    torch.cuda.current_stream().wait_stream(side)
    p2 = PagedQ8(t, [min(n + 5, (n + 15) // 16 * 16) for n in s], 8, 2, 16, 197, max_kv=600)
    assert p2.kq.shape == p.kq.shape and p2.table.shape == p.table.shape
    for a, b in ((p.q, p2.q), (p.kq, p2.kq), (p.vq, p2.vq), (p.sc, p2.sc), (p.table, p2.table),
                 (p.s_d, p2.s_d)):
        a.copy_(b)
    p.rows, p.s = p2.rows, p2.s
    p.o.fill_(-7)
    p.L.fill_(-7)
    p.ws.fill_(math.nan)
    g.replay()
    torch.cuda.synchronize()
    assert pu.status() == 0
    p.check()


@pytest.mark.parametrize("t", [1, 30])
def test_two_calls_at_once(t):
    """Two calls on two streams with a workspace each."""
    ps = [PagedQ8([t] * 4, [4000, 30, 1000, 512], 8, 2, 16, 199 + i) for i in range(2)]
    ss = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s in zip(ps, ss):
            p.run(stream=s)
    torch.cuda.synchronize()
    assert pu.status() == 0
    for p in ps:
        p.check()


@pytest.mark.parametrize("t", [1, 4, 40])
def test_pool_beyond_32_bit_offsets(t):
    """Pages whose elements lie beyond 2^32 of the pool's start."""
    Hq, Hkv, page, s = 16, 8, 16, 100
    pages = 2 ** 32 // (Hkv * page * D) + 64
    p = PagedQ8([t], [s], Hq, Hkv, page, 203)
    big = [torch.zeros(pages, *x.shape[1:], dtype=torch.uint8, device="cuda")
           for x in (p.kq, p.vq, p.sc)]
    n = p.kq.shape[0]
    for x, y in zip(big, (p.kq, p.vq, p.sc)):
        x[-n:] = y
    p.kq, p.vq, p.sc = big
    p.table += pages - n
    p.table.clamp_(max=pages - 1)
    p.cache = q8.cache_of(p.kq, p.vq, p.sc, p.table, p.s_d)
    p.run()
    assert pu.status() == 0
    p.check()
    ko = torch.empty(s, Hkv, D, dtype=torch.bfloat16, device="cuda")
    gqa.gqa_paged_read_q8(p.cache, pu.i32([0, s]), 1, s, ko, Hkv * D, None, 0)
    assert torch.equal(ko, q8.values(*p.rows[0][:2]).to(torch.bfloat16))


# ---- a run of them together -----------------------------------------------------------------------

@pytest.mark.parametrize("window", [0, 48])
def test_steps_over_an_8_bit_cache(window):
    """Two sequences grow in a prompt chunk, further chunks, drafts and single tokens, append then
    attention each time; every output is attention over the numbers that the cache holds, which
    the read-back returns, and those are the keys of one bf16 pass, rounded."""
    Hq, Hkv, page, N = 8, 2, 16, [230, 150]
    gen = _gen(210)
    eps = 1e-6
    xs = [_randn(gen, n, (Hq + 2 * Hkv) * D) for n in N]
    gq, gk = (1 + 0.1 * torch.randn(D, generator=gen)).cuda(), torch.ones(D, device="cuda")
    tab = _table(D, 256)
    row = (Hq + 2 * Hkv) * D
    steps = [(100, 0), (100, 64), (3, 5), (1, 1), (1, 0), (0, 2), (25, 78)]
    kq, vq, sc, table = q8.pools(2, N, Hkv, page, D, gen)
    got, queries, done = [[], []], [[], []], [0, 0]
    for ts in steps:
        x = torch.cat([xs[i][done[i]:done[i] + ts[i]] for i in range(2)])
        done = [a + b for a, b in zip(done, ts)]
        total, cu, lens = x.shape[0], pu.i32(pu.cu_of(ts)), pu.i32(done)
        q, k, v = x.split([Hq * D, Hkv * D, Hkv * D], 1)
        qr = torch.empty(total, Hq, D, dtype=torch.bfloat16, device="cuda")
        o = torch.empty_like(qr)
        cache = q8.cache_of(kq, vq, sc, table, lens)
        gqa.gqa_packed_rope_append_q8(q, row, k, row, v, row, cu, 2, total, Hq, Hkv, D, gq, gk, eps,
                                      tab, 256, qr, None, cache)
        a = (2, total, max(ts), max(done), Hq, Hkv, D)
        wsb = gqa.gqa_attn_paged_q8_workspace_bytes(*a)
        ws = torch.full((max(wsb, 16) // 4 + 1,), math.nan, device="cuda")
        gqa.gqa_attn_paged_q8(qr, Hq * D, cache, cu, 2, total, max(ts), max(done), Hq, window,
                              D ** -0.5, o, Hq * D, None, ws, wsb)
        assert pu.status() == 0
        for i, part in enumerate((slice(0, ts[0]), slice(ts[0], total))):
            got[i].append(o[part])
            queries[i].append(qr[part])
    assert done == N
    # what the cache holds
    total, cu = sum(N), pu.i32(pu.cu_of(N))
    ko = torch.empty(total, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)
    lens = pu.i32(N)
    gqa.gqa_paged_read_q8(q8.cache_of(kq, vq, sc, table, lens), cu, 2, total, ko, Hkv * D, vo,
                          Hkv * D)
    assert pu.status() == 0
    x = torch.cat(xs)
    _, k, v = x.split([Hq * D, Hkv * D, Hkv * D], 1)
    kr = torch.empty(total, Hkv, D, dtype=torch.bfloat16, device="cuda")
    gqa.gqa_packed_rope_append(None, 0, k, row, None, 0, cu, 2, total, 0, Hkv, D, None, gk, eps,
                               tab, 256, None, kr, None)
    assert torch.equal(vo, q8.values(*q8.quantise(v.reshape(total, Hkv, D))).to(torch.bfloat16))
    # two roundings of the same fp32 number: to bf16, and to 4 bits
    step = kr.double().abs().amax(-1, keepdim=True) * 2.0 ** -8
    assert ((ko.double() - kr.double()).abs() <=
            (q8.E4M3 + 2 * pu.BF16) * kr.double().abs() + q8.TINY * step).all()
    at = 0
    for i, n in enumerate(N):
        pg, slot = q8.places(table, i, page, torch.arange(n, device="cuda"))
        ro, _, bo, _ = q8.attention64(torch.cat(queries[i]), kq[pg, :, slot], sc[pg, :, slot, 0],
                                      vq[pg, :, slot], sc[pg, :, slot, 1], window, D ** -0.5)
        pu.check(torch.cat(got[i]), ro, bo, f"steps of sequence {i}")
        at += n
