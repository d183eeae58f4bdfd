"""The packed and paged attention operators: what is timed, and their plain forms.

Three operators of a serving step over packed sequences (tokens of all sequences behind one
another, `cu` holding each sequence's first row):

* ``packed``: causal (or sliding-window) grouped-query attention over whole prompts of
  different lengths;
* ``append``: per-head RMSNorm of q and k, RoPE, and the write of the new tokens' keys and
  values into the pages of a paged cache, from the rows of one fused QKV projection;
* ``paged``: attention of each sequence's new tokens (one when decoding, a few when a draft
  is checked, many in a chunk of a prompt) over all its tokens in the pages.

The head counts are those of the PLaMo 3 31B attention (64 query heads, 8 KV heads of 128)
and smaller or odder ones.
"""
import math
import random

import torch

own = False
D = 128
THETA = 1.0e4
EPS = 1.0e-6


# ---- cases ----------------------------------------------------------------------------------

def _case(name, op, nseq, t, s, hq, hkv, window=0, page=0, norm=False, lens=1):
    """t: range of new tokens per sequence; s: range of tokens already cached (paged ones)."""
    c = {"op": op, "nseq": nseq, "t_lo": t[0], "t_hi": t[1], "s_lo": s[0], "s_hi": s[1],
         "hq": hq, "hkv": hkv, "window": window, "page": page, "norm": norm, "lens": lens}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one short prompt on few heads: a first chat turn on a small model, launch latency
        _case("packed_one_short", "packed", 1, (17, 17), (0, 0), 8, 2),
        # a batch of ordinary prompts, very different lengths, full causal layer
        _case("packed_batch", "packed", 16, (33, 2000), (0, 0), 64, 8),
        # sliding-window layer (self + 2047 earlier) over long prompts of odd lengths
        _case("packed_window", "packed", 4, (2500, 8192), (0, 0), 64, 8, window=2048),
        # the longest prompt, global layer: the compute-bound end
        _case("packed_long", "packed", 1, (16384, 16384), (0, 0), 64, 8),
        # one decode token: the append's launch latency
        _case("append_one", "append", 1, (1, 1), (137, 137), 8, 2, page=16),
        # a decode step's tokens of a large batch, with the q/k norm
        _case("append_decode", "append", 128, (1, 1), (100, 4000), 64, 8, page=16, norm=True),
        # prompts of a prefill step, with the q/k norm
        _case("append_prompt", "append", 8, (300, 4000), (0, 0), 64, 8, page=64, norm=True),
        # one sequence, one token, a short cache
        _case("paged_one", "paged", 1, (1, 1), (137, 137), 8, 2, page=16),
        # decode over long caches, full causal: the bandwidth-bound end
        _case("paged_decode", "paged", 32, (1, 1), (8192, 65535), 64, 8, page=64),
        # decode in a sliding-window layer: every sequence reads its last 2048 tokens
        _case("paged_decode_window", "paged", 64, (1, 1), (1000, 9000), 64, 8, window=2048,
              page=16),
        # drafts of two to four tokens checked in one pass
        _case("paged_draft", "paged", 24, (2, 4), (700, 6000), 32, 8, page=32),
        # a mixed step: long chunks of prompts over what is cached already
        _case("paged_chunk", "paged", 4, (700, 2048), (0, 12000), 64, 8, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["packed", "packed", "append", "paged", "paged", "paged"])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8, 8, 16])
    while hkv * g > 64:
        g = rng.choice([1, 2, 3, 4, 6, 8])
    window = rng.choice([0, 0, _log(rng, 16, 4096)])
    page = rng.choice([16, 32, 64, 128])
    lens = rng.randrange(1, 1 << 20)
    if op == "packed":
        nseq = _log(rng, 1, 48)
        hi = max(2, _log(rng, 2, min(16000, 24000 // nseq + 64)))
        lo = max(1, _log(rng, 1, hi))
        return _case("", op, nseq, (lo, hi), (0, 0), hkv * g, hkv, window=window, lens=lens)
    if op == "append":
        nseq = _log(rng, 1, 128)
        hi = _log(rng, 1, 16000 // nseq + 1)
        return _case("", op, nseq, (max(1, hi // 3), hi), (0, _log(rng, 1, 4000)), hkv * g, hkv,
                     page=page, norm=rng.random() < 0.5, lens=lens)
    kind = rng.choice(["decode", "decode", "draft", "chunk"])
    if kind == "chunk":
        nseq = _log(rng, 1, 8)
        hi = _log(rng, 16, 6000 // nseq)
        t = (1, hi)
        s_hi = _log(rng, 16, 16000)
    else:
        nseq = _log(rng, 1, 64)
        t = (1, 1) if kind == "decode" else (1, rng.randrange(2, 9))
        s_hi = _log(rng, 16, min(60000, 800000 // nseq))
    return _case("", op, nseq, t, (max(0, s_hi // 8), s_hi), hkv * g, hkv, window=window,
                 page=page, lens=lens)


def _lengths(case):
    """(new tokens, all tokens) of each sequence: part of the case, not of the inputs."""
    r = random.Random(case["lens"])
    t = [_log(r, case["t_lo"], case["t_hi"]) for _ in range(case["nseq"])]
    t[0] = case["t_hi"]
    if case["op"] == "packed":
        return t, list(t)
    s = [r.randint(case["s_lo"], case["s_hi"]) for _ in range(case["nseq"])]
    s[-1] = case["s_hi"]
    return t, [a + b for a, b in zip(t, s)]


# ---- what a user's program has in hand ------------------------------------------------------

def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 2 + 1)
    t, s = _lengths(case)
    nseq, hq, hkv, total = case["nseq"], case["hq"], case["hkv"], sum(t)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    cu = [0]
    for n in t:
        cu.append(cu[-1] + n)
    st = {"case": case, "t": t, "s": s, "total": total,
          "cu": torch.tensor(cu, dtype=torch.int32, device="cuda")}
    # one row per token of the fused projection: q heads, k heads, v heads
    st["qkv"] = normal(total, (hq + 2 * hkv) * D)
    if case["op"] != "packed":
        ps = case["page"]
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
        st["k"] = normal(pages, hkv, ps, D)
        st["v"] = normal(pages, hkv, ps, D)
    if case["op"] == "append":
        st["q_gamma"] = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")) if case["norm"] else None
        st["k_gamma"] = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")) if case["norm"] else None
        p = torch.arange(max(s), dtype=torch.float64, device="cuda")
        w = THETA ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
        a = p[:, None] * w
        st["table"] = torch.stack([a.cos(), a.sin()], -1).float().contiguous()   # [pos, D/2, 2]
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    t, s, total, hq, hkv = st["t"], st["s"], st["total"], case["hq"], case["hkv"]
    st["scale"] = D ** -0.5
    row = (hq + 2 * hkv) * D
    st["row"] = row
    st["q"], st["kn"], st["vn"] = st["qkv"].split([hq * D, hkv * D, hkv * D], 1)
    st["out"] = torch.empty(total, hq, D, dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.empty(hq, total, dtype=torch.float32, device="cuda")
    st["rows"] = torch.tensor([i for i, n in enumerate(t) for _ in range(n)], device="cuda")
    st["local"] = torch.tensor([j for n in t for j in range(n)], device="cuda")
    if own:
        import global_causal_gqa_gb300 as gqa
        st["gqa"] = gqa
        if case["op"] != "packed":
            st["cache"] = gqa.make_paged_kv(st["k"], st["v"], st["pages"], st["kv_lens"])
        if case["op"] == "paged":
            st["max_q"], st["max_kv"] = max(t), max(s)
            n = gqa.gqa_attn_paged_workspace_bytes(case["nseq"], total, max(t), max(s), hq, hkv, D)
            st["ws_bytes"] = n
            st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return st


# ---- the plain forms ------------------------------------------------------------------------

def _attend(q, k, v, t, s, window, scale):
    """q [n, T, hkv, g, D], k, v [n, S, hkv, D], padded, with t and s tokens of each sequence:
    a dense masked softmax in 32 bits.  Heads go in slabs that keep the scores below 6 GB."""
    n, T, hkv, g, _ = q.shape
    S = k.shape[1]
    t, s = t.view(n, 1, 1), s.view(n, 1, 1)
    i = s - t + torch.arange(T, device=q.device).view(1, T, 1)
    j = torch.arange(S, device=q.device).view(1, 1, S)
    see = (j <= i) & (j < s)
    if window > 0:
        see &= i - j < window
    see = see[:, None, None]
    step = max(1, min(hkv, int(6e9 / (4.0 * n * g * T * S))))
    out, lse = [], []
    for h in range(0, hkv, step):
        qq = q[:, :, h:h + step].permute(0, 2, 3, 1, 4).float()          # n h g T D
        kk = k[:, :, h:h + step].permute(0, 2, 3, 1).float().unsqueeze(2)  # n h 1 D S
        vv = v[:, :, h:h + step].permute(0, 2, 1, 3).float().unsqueeze(2)  # n h 1 S D
        x = torch.matmul(qq.reshape(n, -1, 1, g * T, D), kk).view(n, -1, g, T, S)
        x = (x * scale).masked_fill_(~see, -math.inf)
        m = x.amax(-1, keepdim=True).nan_to_num_(neginf=0.0)
        x = x.sub_(m).exp_()
        z = x.sum(-1, keepdim=True)
        o = torch.matmul(x.view(n, -1, 1, g * T, S), vv).view(n, -1, g, T, D) / z
        out.append(o.permute(0, 3, 1, 2, 4))
        lse.append((m + z.log()).squeeze(-1).permute(0, 3, 1, 2))
    return torch.cat(out, 2), torch.cat(lse, 2)


def _pad(x, st, T):
    y = x.new_zeros(st["case"]["nseq"], T, *x.shape[1:])
    y[st["rows"], st["local"]] = x
    return y


def _plain_attention(st):
    c = st["case"]
    hq, hkv, n = c["hq"], c["hkv"], c["nseq"]
    T = max(st["t"])
    t = st["cu"][1:] - st["cu"][:-1]
    q = _pad(st["q"].reshape(-1, hkv, hq // hkv, D), st, T)
    if c["op"] == "packed":
        s = t
        k = _pad(st["kn"].reshape(-1, hkv, D), st, T)
        v = _pad(st["vn"].reshape(-1, hkv, D), st, T)
    else:
        s = st["kv_lens"]
        k = st["k"][st["pages"].long()].transpose(2, 3).reshape(n, -1, hkv, D)
        v = st["v"][st["pages"].long()].transpose(2, 3).reshape(n, -1, hkv, D)
    o, lse = _attend(q, k, v, t, s, c["window"], st["scale"])
    o = o[st["rows"], st["local"]].reshape(-1, hq, D).to(torch.bfloat16)
    return o, lse[st["rows"], st["local"]].reshape(-1, hq).t().contiguous()


def _norm_rotate(x, gamma, cs):
    x = x.float()
    if gamma is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma
    a, b = x[..., :D // 2], x[..., D // 2:]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.cat([a * c - b * s, a * s + b * c], -1).to(torch.bfloat16)


def _plain_append(st):
    c = st["case"]
    hq, hkv, ps = c["hq"], c["hkv"], c["page"]
    t = st["cu"][1:] - st["cu"][:-1]
    pos = (st["kv_lens"] - t)[st["rows"]] + st["local"]
    cs = st["table"][pos]
    q = _norm_rotate(st["q"].reshape(-1, hq, D), st["q_gamma"], cs)
    k = _norm_rotate(st["kn"].reshape(-1, hkv, D), st["k_gamma"], cs)
    page, slot = st["pages"][st["rows"], pos // ps].long(), pos % ps
    st["k"][page, :, slot] = k
    st["v"][page, :, slot] = st["vn"].reshape(-1, hkv, D)
    return q, st["k"], st["v"]


# ---- one pass ---------------------------------------------------------------------------------

def run(st):
    c = st["case"]
    if not own:
        return _plain_append(st) if c["op"] == "append" else _plain_attention(st)
    gqa, row, n, total, hq, hkv = st["gqa"], st["row"], c["nseq"], st["total"], c["hq"], c["hkv"]
    if c["op"] == "packed":
        gqa.gqa_attn_packed(st["q"], row, st["kn"], row, st["vn"], row, st["out"], hq * D,
                            st["lse"], st["cu"], n, total, hq, hkv, D, c["window"], st["scale"])
        return st["out"], st["lse"]
    if c["op"] == "append":
        gqa.gqa_packed_rope_append(st["q"], row, st["kn"], row, st["vn"], row, st["cu"], n, total,
                                   hq, hkv, D, st["q_gamma"], st["k_gamma"], EPS, st["table"],
                                   st["table"].shape[0], st["out"], None, st["cache"])
        return st["out"], st["k"], st["v"]
    gqa.gqa_attn_paged(st["q"], row, st["cache"], st["cu"], n, total, st["max_q"], st["max_kv"],
                       hq, c["window"], st["scale"], st["out"], hq * D, st["lse"], st["ws"],
                       st["ws_bytes"])
    return st["out"], st["lse"]


# ---- what a pass cannot do without ------------------------------------------------------------

def work(case):
    t, s = _lengths(case)
    hq, hkv, w, total = case["hq"], case["hkv"], case["window"], sum(t)
    if case["op"] == "append":
        bytes_ = 2 * total * (hq + 2 * hkv) * D * 2 + total * (4 * D + 4) + 8 * case["nseq"]
        return {"bytes": bytes_, "flops": total * (hq + hkv) * D * (3 + (4 if case["norm"] else 0))}
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
    bytes_ = 2 * total * hq * D * 2 + keys * hkv * D * 4 + total * hq * 4 + 4 * case["nseq"]
    return {"bytes": bytes_, "flops": 4 * D * hq * pairs}


# ---- the definition in 64 bits ----------------------------------------------------------------

def _exact_attention(case, st):
    hq, hkv, w = case["hq"], case["hkv"], case["window"]
    g = hq // hkv
    out = torch.empty(st["total"], hq, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(hq, st["total"], dtype=torch.float64, device="cuda")
    at = 0
    for n, (a, b) in enumerate(zip(st["t"], st["s"])):
        rows = st["qkv"][at:at + a].double().view(a, hq + 2 * hkv, D)
        if case["op"] == "packed":
            keys, vals = rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        else:
            ps = case["page"]
            j = torch.arange(b, device="cuda")
            pg = st["pages"][n].long()[j // ps]
            keys, vals = st["k"][pg, :, j % ps].double(), st["v"][pg, :, j % ps].double()
        for h in range(hq):
            kh, vh = keys[:, h // g], vals[:, h // g]
            for lo in range(0, a, 4096):
                hi = min(a, lo + 4096)
                # keys that some query of this block sees
                k1, k0 = b - a + hi, max(0, b - a + lo - w + 1) if w > 0 else 0
                i = b - a + torch.arange(lo, hi, device="cuda")[:, None]
                j = torch.arange(k0, k1, device="cuda")[None]
                x = rows[lo:hi, h] @ kh[k0:k1].T / math.sqrt(D)
                x[(j > i) | ((i - j >= w) if w > 0 else (j > i))] = -math.inf
                z = torch.logsumexp(x, 1)
                lse[h, at + lo:at + hi] = z
                out[at + lo:at + hi, h] = torch.exp(x - z[:, None]) @ vh[k0:k1]
        at += a
    return out, lse


def _exact_append(case, st):
    hq, hkv, ps = case["hq"], case["hkv"], case["page"]
    rows = st["qkv"].double().view(-1, hq + 2 * hkv, D)
    x = rows[:, :hq + hkv]
    if case["norm"]:
        gain = torch.cat([st["q_gamma"].expand(hq, D), st["k_gamma"].expand(hkv, D)]).double()
        x = gain * x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS)
    pos = torch.tensor([b - a + i for a, b in zip(st["t"], st["s"]) for i in range(a)],
                       dtype=torch.float64, device="cuda")
    w = torch.exp(torch.arange(D // 2, dtype=torch.float64, device="cuda") * (-2 * math.log(THETA) / D))
    z = torch.complex(x[..., :D // 2], x[..., D // 2:]) * torch.exp(1j * pos[:, None] * w)[:, None]
    x = torch.cat([z.real, z.imag], -1)
    seq = torch.repeat_interleave(torch.arange(case["nseq"], device="cuda"),
                                  torch.tensor(st["t"], device="cuda"))
    p = pos.long()
    k, v = st["k"].double(), st["v"].double()
    pg = st["pages"].long()[seq, p // ps]
    k[pg, :, p % ps] = x[:, hq:]
    v[pg, :, p % ps] = rows[:, hq + hkv:]
    return x[:, :hq], k, v


def exact(case, seed):
    if case["op"] == "append":
        return _exact_append(case, _inputs(case, seed))
    # 64-bit products of every block: about 1 TFLOP/s
    t, s = _lengths(case)
    if sum(4 * D * case["hq"] * a * b for a, b in zip(t, s)) > 1.0e13:
        return None
    return _exact_attention(case, _inputs(case, seed))
