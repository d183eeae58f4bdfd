"""PagedStack: a step over several layers' paged caches, eagerly and as a replayed graph, against
plain 64-bit forms layer by layer."""
import pytest
import torch

import gpu_utils as gu
import packed_utils as pu

pytestmark = pytest.mark.gpu
D, HQ, HKV, PAGE, EPS = 128, 16, 2, 16, 1e-6


def _stack(t, s, windows, seed, max_q, max_kv):
    import global_causal_gqa_gb300 as gqa
    from global_causal_gqa_gb300.model_step import PagedLayer, PagedStack
    gen = torch.Generator().manual_seed(seed)
    total, width = sum(t), -(-max_kv // PAGE)
    pages = len(t) * width
    table = torch.randperm(pages, generator=gen).to(torch.int32).reshape(len(t), width).cuda()
    layers = []
    for w in windows:
        theta = 1e4 if w else 1e6
        tab = torch.empty(max_kv * D, dtype=torch.float32, device="cuda")
        gqa.gqa_rope_table_build(tab, gqa.gqa_rope_inv_freq(D, theta), D, 1.0, max_kv)
        rnd = lambda *n: torch.randn(*n, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
        layers.append(PagedLayer(rnd(pages, HKV, PAGE, D), rnd(pages, HKV, PAGE, D),
                                 rnd(total, (HQ + 2 * HKV) * D),
                                 torch.zeros(total, HQ, D, dtype=torch.bfloat16, device="cuda"),
                                 (1 + 0.1 * torch.randn(D, generator=gen)).cuda(),
                                 (1 + 0.1 * torch.randn(D, generator=gen)).cuda(), tab, max_kv, w))
    cu, lens = pu.i32(pu.cu_of(t)), pu.i32(s)
    return PagedStack(layers, cu, lens, table, max_q, max_kv, HQ, HKV, D, D ** -0.5, EPS)


def _check(stack, before, t, s):
    """The layers' outputs and pools against the plain forms, from the pools `before` the step.
    The bf16 queries and keys that the append wrote are checked against 64 bits and then feed
    the attention's reference."""
    import global_causal_gqa_gb300 as gqa
    cu = pu.cu_of(t)
    for L, (k0, v0) in zip(stack.layers, before):
        rows = L.qkv.reshape(-1, HQ + 2 * HKV, D)
        theta = 1e4 if L.window else 1e6
        # this layer's queries, from the same call over copies of the pools
        q = torch.empty(rows.shape[0], HQ, D, dtype=torch.bfloat16, device="cuda")
        row = (HQ + 2 * HKV) * D
        xq, xk, xv = L.qkv.split([HQ * D, HKV * D, HKV * D], 1)
        kp, vp = k0.clone(), v0.clone()
        cache = gqa.make_paged_kv(kp, vp, stack.page_table, stack.kv_lens)
        gqa.gqa_packed_rope_append(xq, row, xk, row, xv, row, stack.cu_seqlens, len(t),
                                   rows.shape[0], HQ, HKV, D, L.q_gamma, L.k_gamma, EPS, L.table,
                                   L.table_len, q, None, cache)
        assert pu.status() == 0
        assert torch.equal(kp, L.k_pool) and torch.equal(vp, L.v_pool)
        for i, (a, b) in enumerate(zip(t, s)):
            if a == 0:
                continue
            x = rows[cu[i]:cu[i + 1]]
            j = torch.arange(b, device="cuda")
            pg = stack.page_table[i].long()[j // PAGE]
            pos = torch.arange(b - a, b, device="cuda")
            k, v = L.k_pool[pg, :, j % PAGE], L.v_pool[pg, :, j % PAGE]
            assert torch.equal(k[:b - a], k0[pg, :, j % PAGE][:b - a])
            assert torch.equal(v[:b - a], v0[pg, :, j % PAGE][:b - a])
            assert torch.equal(v[b - a:], x[:, HQ + HKV:])
            for got, ref in ((k[b - a:], pu.rope64(x[:, HQ:HQ + HKV], pos, theta, L.k_gamma, EPS)),
                             (q[cu[i]:cu[i + 1]], pu.rope64(x[:, :HQ], pos, theta, L.q_gamma, EPS))):
                # one rounding to bf16; before it fp32 ones of the table, the norm's D squares
                # and the products, of a pair's length
                pair = torch.cat([ref[..., :D // 2].abs() + ref[..., D // 2:].abs()] * 2, -1)
                pu.check(got, ref, pu.BF16 * ref.abs() + (16 + D) * pu.FP32 * 1.5 * pair, "rotated")
            ro, _, bo, _ = pu.attention64(q[cu[i]:cu[i + 1]], k, v, L.window, D ** -0.5)
            pu.check(L.o[cu[i]:cu[i + 1]], ro, bo, f"o of sequence {i}")


def _pools(stack):
    return [(L.k_pool.clone(), L.v_pool.clone()) for L in stack.layers]


@pytest.mark.parametrize("t,s", [([1, 1, 1], [300, 40, 1]), ([4, 2, 3], [300, 40, 3]),
                                 ([130, 1, 0, 70], [200, 300, 7, 70])])
def test_step_over_layers(t, s):
    gu.require_gpu()
    stack = _stack(t, s, (64, 0, 16), 301 + len(t), max(t), 320)
    before = _pools(stack)
    stack.step()
    assert pu.status() == 0
    _check(stack, before, t, s)


def test_captured_steps_follow_the_lengths():
    """A decode step captured once and replayed while the sequences grow, against eager steps."""
    gu.require_gpu()
    t, s = [1, 1, 1, 1], [30, 200, 1, 64]
    a = _stack(t, s, (64, 0), 311, 1, 320)
    b = _stack(t, s, (64, 0), 311, 1, 320)
    a.step()
    torch.cuda.synchronize()
    graph = a.capture()
    for n in range(3):
        for stack in (a, b):
            stack.kv_lens.copy_(pu.i32([x + 7 * n for x in s]))
            for L in stack.layers:
                L.o.zero_()
        graph.replay()
        b.step()
        torch.cuda.synchronize()
        assert pu.status() == 0
        for L, M in zip(a.layers, b.layers):
            assert torch.equal(L.o, M.o) and torch.equal(L.k_pool, M.k_pool)
