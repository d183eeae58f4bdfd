"""Plain 64-bit forms of the 8-bit paged cache, and the error bounds of attention over it."""
import math

import torch

import global_causal_gqa_gb300 as gqa
import packed_utils as pu

E4M3 = 2.0 ** -4          # half a step of a normal e4m3 number, relative to the value
TINY = 2.0 ** -10         # half a step below 2^-6
E_LO, E_HI = -126, 119


def power(byte):
    """2^(byte - 127) in 64 bits; NaN for 255."""
    e = byte.double() - 127
    return torch.where(byte == 255, math.nan, torch.exp2(e))


def scale_bytes(most):
    """The byte of vectors whose largest magnitude is `most` (64 bits)."""
    frac, ex = torch.frexp(torch.where(torch.isfinite(most), most, 1.0))
    e = (ex - 9 + (frac > 0.875).int()).clamp(E_LO, E_HI)
    e = torch.where(most == 0, E_LO, e)
    return torch.where(torch.isfinite(most), e + 127, 255).to(torch.uint8)


def quantise(x):
    """x [..., d] -> (e4m3 numbers as uint8, scale bytes [...])."""
    x = x.double()
    byte = scale_bytes(x.abs().amax(-1))
    y = (x / torch.exp2(byte.double() - 127)[..., None]).clamp(-448, 448)
    y = torch.where((byte == 255)[..., None], torch.zeros_like(y), y)
    return y.float().to(torch.float8_e4m3fn).view(torch.uint8), byte


def numbers(data):
    return data.view(torch.float8_e4m3fn).double()


def values(data, byte):
    return numbers(data) * power(byte)[..., None]


def attention64(q, kd, kb, vd, vb, window, scale):
    """packed_utils.attention64 over a sequence's numbers and bytes [S, Hkv, ...].  Besides the
    roundings named there (a weight to bf16: 2^-8; as a sum of three e5m2 numbers of an f16 it is
    off by 2^-9 + 2^-11) a kernel may bring q to two e4m3 numbers with the row's largest element
    between 2^7 and 2^8, h + l / 16: exact above 2^-3; below, l / 16 is a multiple of 2^-13, an
    element is off by 2^-14 at most, 2^-21 of the largest.  And a weight times its value's power of
    two is such a sum with the row's largest product between 2^12 and 2^15, and loses at most 2^-17
    of it, 2^-29 of the largest."""
    S = kd.shape[0]
    k, v = values(kd, kb), values(vd, vb)
    o, lse, bo, bl = pu.attention64(q, k, v, window, scale)
    T, Hq, _ = q.shape
    G = Hq // kd.shape[1]
    i = torch.arange(S - T, S, device=q.device)[:, None]
    j = torch.arange(S, device=q.device)[None]
    see = (j <= i) & ((i - j < window) if window > 0 else (j <= i))
    for h in range(Hq):
        g = h // G
        r = scale * 2.0 ** -21 * q[:, h].double().abs().amax(1) * k[:, g].abs().sum(1).max()
        p = torch.exp(scale * (q[:, h].double() @ k[:, g].T) - lse[h][:, None])
        p = torch.where(see, p, 0.0)
        bl[h] += r
        bo[:, h] += 2 * r[:, None] * (p @ v[:, g].abs())
        most = (p * torch.where(see, power(vb[:, g]), 0.0)).amax(1)
        bo[:, h] += 2.0 ** -29 * most[:, None] * (see.double() @ numbers(vd[:, g]).abs())
    return o, lse, bo, bl


def pools(nseq, lens, Hkv, page, d, gen, spare=3):
    """Pools whose every number and byte is NaN, and a page table as packed_utils.pools gives."""
    k, _, table = pu.pools(nseq, lens, Hkv, page, d, gen, spare)
    n = k.shape[0]
    kq = torch.full((n, Hkv, page, d), 0x7f, dtype=torch.uint8, device="cuda")
    sc = torch.full((n, Hkv, page, 2), 255, dtype=torch.uint8, device="cuda")
    return kq, kq.clone(), sc, table


def cache_of(kq, vq, sc, table, lens):
    a = gqa.make_paged_kv_q8(kq.view(torch.float8_e4m3fn), vq.view(torch.float8_e4m3fn),
                             sc.view(torch.float8_e8m0fnu), table, lens)
    a.keep = (kq, vq, sc, table, lens)     # the struct holds addresses only
    return a


def places(table, i, page, j):
    """(page, slot) of positions j of sequence i."""
    return table[i].long()[j // page], j % page
