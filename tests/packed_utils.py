"""Plain 64-bit forms of the packed and paged operators, and the error bounds of their bf16
results, for the GPU tests."""
import math

import numpy as np
import torch

import global_causal_gqa_gb300 as gqa

# A rounding to bf16 is off by at most half a step, 2^-8 of the value; fp32 by 2^-24.
BF16, FP32 = 2.0 ** -8, 2.0 ** -24


def cu_of(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def attention64(q, k, v, window, scale):
    """One sequence in 64 bits: q [T, Hq, d], k, v [S, Hkv, d].  Returns (o, lse, bound_o,
    bound_lse), o [T, Hq, d], lse [Hq, T].

    The bounds.  A kernel forms the scores from exact products of bf16 values with an fp32
    sum of d terms: off by at most 2 d 2^-24 scale sum_i |q_i k_i| =: e (2: a tensor core may
    truncate instead of round), plus the argument's and the exponential's own error, within
    2^-22 (2 + |x| log2 e) of a weight.  Let r be the relative error of a weight before it
    meets V: r <= 2 e + 2^-20 (2 + |x|).  The weights are rounded to bf16 (BF16 each) against
    an unrounded fp32 sum, and the result once more:
    |o' - o| <= (BF16 + 2 r) sum_j p_j |v_j| + BF16 |o| (1 + BF16), and lse is off by at most
    r + 2^-22 |lse|."""
    T, Hq, d = q.shape
    S, Hkv, _ = k.shape
    G = Hq // Hkv
    q, k, v = q.double(), k.double(), v.double()
    i = torch.arange(S - T, S, device=q.device)[:, None]
    j = torch.arange(S, device=q.device)[None]
    hide = j > i
    if window > 0:
        hide = hide | (i - j >= window)
    o = torch.empty(T, Hq, d, dtype=torch.float64, device=q.device)
    lse = torch.empty(Hq, T, dtype=torch.float64, device=q.device)
    bo, bl = torch.empty_like(o), torch.empty_like(lse)
    for h in range(Hq):
        g = h // G
        x = scale * (q[:, h] @ k[:, g].T)
        ax = scale * (q[:, h].abs() @ k[:, g].abs().T)
        x = x.masked_fill(hide, -math.inf)
        ax = ax.masked_fill(hide, 0.0)
        z = torch.logsumexp(x, 1)
        p = torch.exp(x - z[:, None])
        # a hidden key's value has no part in the result, whatever it is
        seen = ~hide.all(0)
        vv = torch.where(seen[:, None], v[:, g], torch.zeros_like(v[:, g]))
        o[:, h] = p @ vv
        lse[h] = z
        r = 2 * 2 * d * FP32 * ax.amax(1) + 2.0 ** -20 * (2 + ax.amax(1))
        bo[:, h] = (BF16 + 2 * r)[:, None] * (p @ vv.abs()) + BF16 * (1 + BF16) * o[:, h].abs()
        bl[h] = r + 2.0 ** -22 * z.abs()
    return o, lse, bo, bl


def rope64(x, pos, theta, gamma=None, eps=0.0, amp=1.0):
    """x [n, H, d] -> amp * rotation of N(x) at pos [n], in 64 bits."""
    d = x.shape[-1]
    x = x.double()
    if gamma is not None:
        x = gamma.double() * x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    w = theta ** (-torch.arange(0, d, 2, dtype=torch.float64, device=x.device) / d)
    a = pos.double()[:, None] * w
    c, s = (amp * a.cos())[:, None], (amp * a.sin())[:, None]
    x0, x1 = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([x0 * c - x1 * s, x0 * s + x1 * c], -1)


def check(got, want, bound, what):
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    bad = err > bound
    if bad.any():
        at = int((err / bound.clamp_min(1e-300)).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {err.numel()} beyond the bound, worst "
                             f"{err.flatten()[at]:.3e} against {bound.flatten()[at]:.3e}")


def pools(nseq, lens, Hkv, page, d, gen, spare=3, fill=math.nan):
    """Empty pools (filled with `fill`), and a page table in random order whose unused entries
    point far outside the pool."""
    per = [-(-n // page) for n in lens]
    pages, width = sum(per) + spare, max(1, max(per))
    perm = torch.randperm(pages, generator=gen).to(torch.int32)
    table = torch.full((nseq, width), 2 ** 31 - 1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = perm[at:at + n]
        at += n
    k = torch.full((pages, Hkv, page, d), fill, dtype=torch.bfloat16, device="cuda")
    return k, k.clone(), table.cuda()


def put(pool, table, i, rows):
    """rows [S, Hkv, d] of sequence i into its pages."""
    page = pool.shape[2]
    j = torch.arange(rows.shape[0], device="cuda")
    pool[table[i].long()[j // page], :, j % page] = rows


def status():
    return gqa.gqa_get_device_status()


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")
