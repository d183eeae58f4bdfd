"""The operators of the 8-bit paged cache: what is timed, and their plain forms.

The cache keeps each key and value vector (one token, one KV head) as d e4m3 numbers and one
power of two, 2^e with the smallest e for which max |x| <= 448 * 2^e:

* ``append``: per-head RMSNorm of q and k, RoPE, and the write of the new tokens' keys and
  values into the pages in that form, from the rows of one fused QKV projection;
* ``paged``: attention of each sequence's new tokens (one when decoding, a few when a draft
  is checked, many in a chunk of a prompt) over all its tokens in the pages;
* ``read``: the last tokens of every sequence read back into packed bfloat16 rows.

The head counts are those of the PLaMo 3 31B attention (64 query heads, 8 KV heads of 128)
and smaller or odder ones; the head dimensions of append and read are also the others that the
framework's caches have (64, 256, 512).
"""
import math
import random

import torch

own = False
THETA = 1.0e4
EPS = 1.0e-6
MOST = 448.0                  # the largest e4m3 number
E_LO, E_HI = -126, 119        # the exponents of a vector's power of two


# ---- cases ----------------------------------------------------------------------------------

def _case(name, op, nseq, t, s, hq, hkv, page, window=0, norm=False, d=128, lens=1):
    """t: range of new tokens per sequence (read: of tokens read); s: range of tokens before
    them."""
    c = {"op": op, "nseq": nseq, "t_lo": t[0], "t_hi": t[1], "s_lo": s[0], "s_hi": s[1],
         "hq": hq, "hkv": hkv, "page": page, "window": window, "norm": norm, "d": d, "lens": lens}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode token: launch latency of the append
        _case("append_one", "append", 1, (1, 1), (137, 137), 8, 2, 16),
        # a decode step's tokens of a large batch, with the q/k norm
        _case("append_decode", "append", 128, (1, 1), (100, 4000), 64, 8, 16, norm=True),
        # prompts of a prefill step, with the q/k norm
        _case("append_prompt", "append", 8, (300, 4000), (0, 0), 64, 8, 64, norm=True),
        # one sequence, one token, a short cache: latency
        _case("paged_one", "paged", 1, (1, 1), (137, 137), 8, 2, 16),
        # decode over many short caches: chats that have just begun
        _case("paged_short", "paged", 256, (1, 1), (20, 450), 32, 8, 16),
        # decode over long caches, full causal: the bandwidth-bound end
        _case("paged_decode", "paged", 32, (1, 1), (8192, 65535), 64, 8, 64),
        # decode in a sliding-window layer: every sequence reads its last 2048 tokens
        _case("paged_decode_window", "paged", 64, (1, 1), (1000, 9000), 64, 8, 16, window=2048),
        # drafts of two to six tokens checked in one pass, with 8 query heads per KV head
        _case("paged_draft", "paged", 24, (2, 6), (700, 6000), 64, 8, 32),
        # a mixed step: long chunks of prompts over what is cached already
        _case("paged_chunk", "paged", 4, (700, 2048), (0, 12000), 64, 8, 16),
        # a few tokens handed to another cache
        _case("read_few", "read", 1, (17, 17), (120, 120), 8, 2, 16),
        # the sequences of a batch leave the cache in an odd number of tokens each
        _case("read_batch", "read", 12, (301, 9001), (0, 500), 64, 8, 32),
        # one long prefix, wide heads
        _case("read_wide", "read", 1, (16001, 16001), (0, 0), 16, 2, 128, d=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "paged", "paged", "paged", "paged", "read"])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8, 8, 16])
    while hkv * g > 64:
        g = rng.choice([1, 2, 3, 4, 6, 8])
    page = rng.choice([16, 32, 64, 128])
    lens = rng.randrange(1, 1 << 20)
    d = rng.choice([64, 128, 128, 128, 256, 512])
    room = 128 * 8 // (d * hkv) if d * hkv <= 1024 else 1   # small vectors: more tokens
    if op == "append":
        nseq = _log(rng, 1, 128)
        hi = _log(rng, 1, 12000 * min(room, 2) // nseq + 1)
        if d > 128:
            hkv, g = min(hkv, 4), min(g, 4)
        return _case("", op, nseq, (max(1, hi // 3), hi), (0, _log(rng, 1, 4000)), hkv * g, hkv,
                     page, norm=rng.random() < 0.5, d=d, lens=lens)
    if op == "read":
        nseq = _log(rng, 1, 64)
        hi = _log(rng, 1, 60000 * min(room, 4) // nseq)
        return _case("", op, nseq, (max(1, hi // 4), hi), (0, _log(rng, 1, 1000)), hkv * g, hkv,
                     page, d=d, lens=lens)
    window = rng.choice([0, 0, _log(rng, 16, 4096)])
    kind = rng.choice(["decode", "decode", "draft", "chunk"])
    if kind == "chunk":
        nseq = _log(rng, 1, 8)
        t = (1, _log(rng, 16, 6000 // nseq))
        s_hi = _log(rng, 16, 16000)
    else:
        nseq = _log(rng, 1, 128)
        t = (1, 1) if kind == "decode" else (1, rng.randrange(2, 9))
        s_hi = _log(rng, 16, min(60000, 800000 // nseq))
    return _case("", op, nseq, t, (max(0, s_hi // 8), s_hi), hkv * g, hkv, page, window=window,
                 lens=lens)


def _lengths(case):
    """(new tokens, all tokens) of each sequence: part of the case, not of the inputs."""
    r = random.Random(case["lens"])
    t = [_log(r, case["t_lo"], case["t_hi"]) for _ in range(case["nseq"])]
    t[0] = case["t_hi"]
    s = [r.randint(case["s_lo"], case["s_hi"]) for _ in range(case["nseq"])]
    s[-1] = case["s_hi"]
    return t, [a + b for a, b in zip(t, s)]


# ---- the 8-bit form -------------------------------------------------------------------------

def _quantise(x):
    """x [..., d] in 64 bits: (e4m3 bytes [..., d], scale bytes [...])."""
    most = x.abs().amax(-1)
    frac, ex = torch.frexp(most)                       # most = frac 2^ex, frac in [0.5, 1)
    e = (ex - 9 + (frac > MOST / 512).int()).clamp(E_LO, E_HI)
    e = torch.where(most == 0, E_LO, e)
    y = torch.ldexp(x, -e[..., None])
    return y.float().to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _power(byte):
    """2^(byte - 127) in 32 bits."""
    return (byte.int() << 23).view(torch.float32)


def _values(data, byte):
    """What e4m3 bytes [..., d] with scale bytes [...] stand for, in 32 bits."""
    return data.view(torch.float8_e4m3fn).float() * _power(byte)[..., None]


# ---- what a user's program has in hand ------------------------------------------------------

def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 2 + 1)
    t, s = _lengths(case)
    nseq, hq, hkv, d, ps, total = (case["nseq"], case["hq"], case["hkv"], case["d"],
                                   case["page"], sum(t))
    cu = [0]
    for n in t:
        cu.append(cu[-1] + n)
    st = {"case": case, "t": t, "s": s, "total": total,
          "cu": torch.tensor(cu, dtype=torch.int32, device="cuda")}
    per = [-(-n // ps) for n in s]
    pages, width = sum(per) + 3, max(per)
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(nseq, width, dtype=torch.int64)
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = torch.arange(at, at + n)
        at += n
    st["pages"] = perm[table.cuda()].contiguous()
    st["kv_lens"] = torch.tensor(s, dtype=torch.int32, device="cuda")
    # normal numbers of a spread of sizes as they are kept: the largest of a vector between 224
    # and 448, its power of two around that of vectors of unit variance
    step = max(1, (1 << 28) // (hkv * ps * d))
    st["scales"] = torch.randint(117, 123, (pages, hkv, ps, 2), generator=g, device="cuda",
                                 dtype=torch.uint8)
    for name in ("k", "v"):
        x = torch.empty(pages, hkv, ps, d, dtype=torch.uint8, device="cuda")
        for lo in range(0, pages, step):
            y = torch.randn(min(step, pages - lo), hkv, ps, d, generator=g, device="cuda")
            x[lo:lo + step] = (y * 96).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        st[name] = x.view(torch.float8_e4m3fn)
    st["scales"] = st["scales"].view(torch.float8_e8m0fnu)
    if case["op"] != "read":
        # one row per token of the fused projection: q heads, k heads, v heads
        st["qkv"] = torch.randn(total, (hq + 2 * hkv) * d, generator=g,
                                device="cuda").to(torch.bfloat16)
    if case["op"] == "append":
        st["q_gamma"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")) if case["norm"] else None
        st["k_gamma"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")) if case["norm"] else None
        p = torch.arange(max(s), dtype=torch.float64, device="cuda")
        w = THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
        a = p[:, None] * w
        st["table"] = torch.stack([a.cos(), a.sin()], -1).float().contiguous()   # [pos, d/2, 2]
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    t, s, total, hq, hkv, d = (st["t"], st["s"], st["total"], case["hq"], case["hkv"], case["d"])
    st["scale"] = d ** -0.5
    st["row"] = (hq + 2 * hkv) * d
    if case["op"] == "read":
        st["k_out"] = torch.empty(total, hkv, d, dtype=torch.bfloat16, device="cuda")
        st["v_out"] = torch.empty(total, hkv, d, dtype=torch.bfloat16, device="cuda")
    else:
        st["q"], st["kn"], st["vn"] = st["qkv"].split([hq * d, hkv * d, hkv * d], 1)
        st["out"] = torch.empty(total, hq, d, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty(hq, total, dtype=torch.float32, device="cuda")
    n = torch.tensor(t, device="cuda")
    st["rows"] = torch.repeat_interleave(torch.arange(case["nseq"], device="cuda"), n)
    st["local"] = torch.arange(total, device="cuda") - st["cu"][:-1].long()[st["rows"]]
    if own:
        import global_causal_gqa_gb300 as gqa
        st["gqa"] = gqa
        st["cache"] = gqa.make_paged_kv_q8(st["k"], st["v"], st["scales"], st["pages"],
                                           st["kv_lens"])
        if case["op"] == "paged":
            st["max_q"], st["max_kv"] = max(t), max(s)
            b = gqa.gqa_attn_paged_q8_workspace_bytes(case["nseq"], total, max(t), max(s), hq,
                                                      hkv, d)
            st["ws_bytes"] = b
            st["ws"] = torch.empty(max(b, 16), dtype=torch.uint8, device="cuda")
    return st


# ---- the plain forms ------------------------------------------------------------------------

def _attend(q, keys, values, t, s, window, scale):
    """q [n, T, hkv, g, D]; keys(h0, h1), values(h0, h1): [n, S, h, D] in 32 bits, padded, with
    t and s tokens of each sequence: a dense masked softmax in 32 bits.  Heads go in slabs that
    keep the scores below 6 GB."""
    n, T, hkv, g, D = q.shape
    S = keys.length
    t, s = t.view(n, 1, 1), s.view(n, 1, 1)
    i = s - t + torch.arange(T, device=q.device).view(1, T, 1)
    j = torch.arange(S, device=q.device).view(1, 1, S)
    see = (j <= i) & (j < s)
    if window > 0:
        see &= i - j < window
    see = see[:, None, None]
    step = max(1, min(hkv, int(6e9 / (4.0 * n * max(g * T, D) * S))))
    out, lse = [], []
    for h in range(0, hkv, step):
        qq = q[:, :, h:h + step].permute(0, 2, 3, 1, 4).float()                # n h g T D
        kk = keys(h, h + step).permute(0, 2, 3, 1)                             # n h D S
        x = torch.matmul(qq.reshape(n, -1, g * T, D), kk).view(n, -1, g, T, S)
        x = (x * scale).masked_fill_(~see, -math.inf)
        m = x.amax(-1, keepdim=True).nan_to_num_(neginf=0.0)
        x = x.sub_(m).exp_()
        z = x.sum(-1, keepdim=True)
        vv = values(h, h + step).permute(0, 2, 1, 3)                           # n h S D
        o = torch.matmul(x.view(n, -1, g * T, S), vv).view(n, -1, g, T, D) / z
        out.append(o.permute(0, 3, 1, 2, 4))
        lse.append((m + z.log()).squeeze(-1).permute(0, 3, 1, 2))
    return torch.cat(out, 2), torch.cat(lse, 2)


class _Pages:
    """The keys (or values) of all sequences, padded, some heads at a time, in 32 bits."""

    def __init__(self, st, name, which):
        self.data, self.byte = st[name].view(torch.uint8), st["scales"].view(torch.uint8)[..., which]
        self.pages = st["pages"].long()
        self.length = self.pages.shape[1] * st["case"]["page"]

    def __call__(self, h0, h1):
        x = _values(self.data[:, h0:h1][self.pages], self.byte[:, h0:h1][self.pages])
        n, w, h, ps, d = x.shape
        return x.transpose(2, 3).reshape(n, w * ps, h, d)


def _plain_attention(st):
    c = st["case"]
    hq, hkv, n, d = c["hq"], c["hkv"], c["nseq"], c["d"]
    x = st["q"].reshape(-1, hkv, hq // hkv, d)
    q = x.new_zeros(n, max(st["t"]), *x.shape[1:])
    q[st["rows"], st["local"]] = x
    o, lse = _attend(q, _Pages(st, "k", 0), _Pages(st, "v", 1), st["cu"][1:] - st["cu"][:-1],
                     st["kv_lens"], c["window"], st["scale"])
    o = o[st["rows"], st["local"]].reshape(-1, hq, d).to(torch.bfloat16)
    return o, lse[st["rows"], st["local"]].reshape(-1, hq).t().contiguous()


def _norm_rotate(x, gamma, cs):
    if gamma is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma
    a, b = x.chunk(2, -1)
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def _places(st):
    """(position, page, slot) of each packed row."""
    ps = st["case"]["page"]
    t = st["cu"][1:] - st["cu"][:-1]
    pos = (st["kv_lens"] - t).long()[st["rows"]] + st["local"]
    return pos, st["pages"].long()[st["rows"], pos // ps], pos % ps


def _plain_append(st):
    c = st["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    pos, page, slot = _places(st)
    cs = st["table"][pos]
    q = _norm_rotate(st["q"].reshape(-1, hq, d).float(), st["q_gamma"], cs).to(torch.bfloat16)
    # what is rounded to 4 bits is computed in 64: it may lie next to a border
    k = _norm_rotate(st["kn"].reshape(-1, hkv, d).double(), st["k_gamma"], cs.double())
    v = st["vn"].reshape(-1, hkv, d).double()
    scales = st["scales"].view(torch.uint8)
    for which, (name, x) in enumerate((("k", k), ("v", v))):
        data, byte = _quantise(x)
        st[name].view(torch.uint8)[page, :, slot] = data
        scales[page, :, slot, which] = byte
    return q, st["k"], st["v"], st["scales"]


def _plain_read(st):
    _, page, slot = _places(st)
    byte = st["scales"].view(torch.uint8)[page, :, slot]
    return tuple(_values(st[name].view(torch.uint8)[page, :, slot], byte[..., i]).to(torch.bfloat16)
                 for i, name in enumerate(("k", "v")))


# ---- one pass ---------------------------------------------------------------------------------

def run(st):
    c = st["case"]
    op, row, n, total, hq, hkv, d = (c["op"], st["row"], c["nseq"], st["total"], c["hq"],
                                     c["hkv"], c["d"])
    if not own:
        return {"append": _plain_append, "paged": _plain_attention, "read": _plain_read}[op](st)
    gqa = st["gqa"]
    if op == "append":
        gqa.gqa_packed_rope_append_q8(st["q"], row, st["kn"], row, st["vn"], row, st["cu"], n,
                                      total, hq, hkv, d, st["q_gamma"], st["k_gamma"], EPS,
                                      st["table"], st["table"].shape[0], st["out"], None,
                                      st["cache"])
        return st["out"], st["k"], st["v"], st["scales"]
    if op == "paged":
        gqa.gqa_attn_paged_q8(st["q"], row, st["cache"], st["cu"], n, total, st["max_q"],
                              st["max_kv"], hq, c["window"], st["scale"], st["out"], hq * d,
                              st["lse"], st["ws"], st["ws_bytes"])
        return st["out"], st["lse"]
    gqa.gqa_paged_read_q8(st["cache"], st["cu"], n, total, st["k_out"], hkv * d, st["v_out"],
                          hkv * d)
    return st["k_out"], st["v_out"]


# ---- what a pass cannot do without ------------------------------------------------------------

def work(case):
    t, s = _lengths(case)
    hq, hkv, w, d, total = case["hq"], case["hkv"], case["window"], case["d"], sum(t)
    if case["op"] == "append":
        bytes_ = total * (2 * (2 * hq + 2 * hkv) * d + 2 * hkv * (d + 1) + 4 * d + 4) + 8 * case["nseq"]
        return {"bytes": bytes_,
                "flops": total * d * ((hq + hkv) * (3 + (4 if case["norm"] else 0)) + 4 * hkv)}
    if case["op"] == "read":
        return {"bytes": total * 2 * hkv * (d + 1 + 2 * d) + 8 * case["nseq"],
                "flops": total * 2 * hkv * d}
    pairs = keys = 0
    for a, b in zip(t, s):
        first = b - a            # position of the first query
        if w > 0:
            # sum over positions p in [first, b) of min(p + 1, w)
            short = max(0, min(b, w) - first)          # positions below w
            lo = min(first, b)
            pairs += short * (2 * lo + short + 1) // 2 + (a - short) * w
            keys += b - max(0, first - w + 1)
        else:
            pairs += a * (first + 1) + a * (a - 1) // 2
            keys += b
    bytes_ = 2 * total * hq * d * 2 + keys * hkv * 2 * (d + 1) + total * hq * 4 + 4 * case["nseq"]
    return {"bytes": bytes_, "flops": 4 * d * hq * pairs}


# ---- the definition in 64 bits ----------------------------------------------------------------

def _stored(st, name, which, page, slot):
    """Vectors of the pool at [page, :, slot], in 64 bits."""
    x = st[name].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).double()
    e = st["scales"].view(torch.uint8)[page, :, slot, which].double() - 127
    return x * torch.exp2(e)[..., None]


def _exact_attention(case, st):
    hq, hkv, w, d, ps = case["hq"], case["hkv"], case["window"], case["d"], case["page"]
    g = hq // hkv
    out = torch.empty(st["total"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(hq, st["total"], dtype=torch.float64, device="cuda")
    at = 0
    for n, (a, b) in enumerate(zip(st["t"], st["s"])):
        q = st["qkv"][at:at + a, :hq * d].double().view(a, hq, d)
        j = torch.arange(b, device="cuda")
        pg = st["pages"][n].long()[j // ps]
        keys, vals = _stored(st, "k", 0, pg, j % ps), _stored(st, "v", 1, pg, j % ps)
        for h in range(hq):
            kh, vh = keys[:, h // g], vals[:, h // g]
            for lo in range(0, a, 4096):
                hi = min(a, lo + 4096)
                # keys that some query of this block sees
                k1, k0 = b - a + hi, max(0, b - a + lo - w + 1) if w > 0 else 0
                i = b - a + torch.arange(lo, hi, device="cuda")[:, None]
                jj = torch.arange(k0, k1, device="cuda")[None]
                x = q[lo:hi, h] @ kh[k0:k1].T / math.sqrt(d)
                x[(jj > i) | ((i - jj >= w) if w > 0 else (jj > i))] = -math.inf
                z = torch.logsumexp(x, 1)
                lse[h, at + lo:at + hi] = z
                out[at + lo:at + hi, h] = torch.exp(x - z[:, None]) @ vh[k0:k1]
        at += a
    return out, lse


def _exact_places(case, st):
    pos = torch.tensor([b - a + i for a, b in zip(st["t"], st["s"]) for i in range(a)],
                       device="cuda")
    seq = torch.repeat_interleave(torch.arange(case["nseq"], device="cuda"),
                                  torch.tensor(st["t"], device="cuda"))
    return pos, st["pages"].long()[seq, pos // case["page"]], pos % case["page"]


def _exact_append(case, st):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    pos, pg, slot = _exact_places(case, st)
    rows = st["qkv"].double().view(-1, hq + 2 * hkv, d)
    x = rows[:, :hq + hkv]
    if case["norm"]:
        gain = torch.cat([st["q_gamma"].expand(hq, d), st["k_gamma"].expand(hkv, d)]).double()
        x = gain * x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS)
    w = torch.exp(torch.arange(d // 2, dtype=torch.float64, device="cuda") * (-2 * math.log(THETA) / d))
    turn = torch.exp(1j * pos.double()[:, None] * w)[:, None]
    z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * turn
    x = torch.cat([z.real, z.imag], -1)
    got = [x[:, :hq]]
    scales = torch.exp2(st["scales"].view(torch.uint8).double() - 127)
    for which, (name, y) in enumerate((("k", x[:, hq:]), ("v", rows[:, hq + hkv:]))):
        pool = st[name].double()
        most = y.abs().amax(-1)
        e = torch.ceil(torch.log2(most / MOST)).clamp(E_LO, E_HI)
        e = torch.where(most <= MOST * torch.exp2(e - 1), e - 1, e)   # the logarithm's rounding
        e = torch.where(most > MOST * torch.exp2(e), e + 1, e)
        pool[pg, :, slot] = y / torch.exp2(e)[..., None]
        scales[pg, :, slot, which] = torch.exp2(e)
        got.append(pool)
    return (*got, scales)


def exact(case, seed):
    if case["op"] == "append":
        return _exact_append(case, _inputs(case, seed))
    if case["op"] == "read":
        st = _inputs(case, seed)
        _, pg, slot = _exact_places(case, st)
        return _stored(st, "k", 0, pg, slot), _stored(st, "v", 1, pg, slot)
    # 64-bit products of every block: about 1 TFLOP/s
    t, s = _lengths(case)
    if sum(4 * case["d"] * case["hq"] * a * b for a, b in zip(t, s)) > 1.0e13:
        return None
    return _exact_attention(case, _inputs(case, seed))
