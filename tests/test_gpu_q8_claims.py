"""Batches that are cut into levels of chunks, which the CTAs claim as they come: the parts of every
output, and their order, are the same whoever takes them."""
import pytest
import torch

import global_causal_gqa_gb300 as gqa
import gpu_utils as gu
import packed_utils as pu
import q8_utils as q8
from test_gpu_packed import D, _gen, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


@pytest.mark.parametrize("Hq,most", [(8, 1), (32, 2), (24, 4), (128, 1), (64, 3), (64, 6)])
@pytest.mark.parametrize("page", [16, 128])
def test_same_bits_whoever_takes_a_chunk(Hq, most, page):
    """60 sequences of 1000 to 9000 tokens over pages that they share (8 KV heads: more than 128
    units per SM); runs with another kernel's blocks in the way, and without."""
    n, Hkv, gen = 60, 8, _gen(900 + Hq + page)
    s = [1000 + (8000 * 7 * i // n) % 8001 for i in range(n)]
    t = [1 + (3 * i) % most for i in range(n)]
    pages = 8192 // page
    kd, kb = q8.quantise(torch.randn(pages, Hkv, page, D, generator=gen).cuda())
    vd, vb = q8.quantise(torch.randn(pages, Hkv, page, D, generator=gen).cuda())
    table = torch.randint(0, pages, (n, (max(s) + page - 1) // page), generator=gen).int().cuda()
    sc = torch.stack([kb, vb], -1).contiguous()
    cache = q8.cache_of(kd, vd, sc, table, pu.i32(s))
    cu, total = pu.cu_of(t, 0), sum(t)
    q = _randn(gen, total, Hq, D)
    a = (n, total, most, max(s), Hq, Hkv, D)
    wsb = gqa.gqa_attn_paged_q8_workspace_bytes(*a)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    cu = pu.i32(cu)
    busy, side = torch.randn(4096, 4096, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for i in range(24):
        o = torch.empty(total, Hq, D, dtype=torch.bfloat16, device="cuda")
        L = torch.empty(Hq, total, device="cuda")
        if i % 3 == 1:
            with torch.cuda.stream(side):
                busy.mul_(1.0)
        gqa.gqa_attn_paged_q8(q, Hq * D, cache, cu, n, total, most, max(s), Hq, 0, D ** -0.5, o,
                              Hq * D, L, ws, wsb)
        torch.cuda.synchronize()
        outs.append((o, L))
    assert pu.status() == 0
    for o, L in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(L, outs[0][1])
