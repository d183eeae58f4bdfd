"""PagedStack with 8-bit layers next to bf16 ones: a step, eagerly and as a replayed graph, against
the calls it is made of and plain 64-bit forms."""
import dataclasses

import pytest
import torch

import global_causal_gqa_gb300 as gqa
import gpu_utils as gu
import packed_utils as pu
import q8_utils as q8
from test_gpu_paged_stack import D, EPS, HKV, HQ, PAGE, _stack as _bf16_stack

pytestmark = pytest.mark.gpu


def _stack(t, s, windows, seed, max_q, max_kv):
    """Every second layer's pools quantised."""
    from global_causal_gqa_gb300.model_step import PagedStack
    a = _bf16_stack(t, s, windows, seed, max_q, max_kv)
    layers = list(a.layers)
    for i in range(0, len(layers), 2):
        L = layers[i]
        (kd, kb), (vd, vb) = q8.quantise(L.k_pool), q8.quantise(L.v_pool)
        layers[i] = dataclasses.replace(
            L, k_pool=kd.view(torch.float8_e4m3fn), v_pool=vd.view(torch.float8_e4m3fn),
            scales=torch.stack([kb, vb], -1).contiguous().view(torch.float8_e8m0fnu))
    return PagedStack(layers, a.cu_seqlens, a.kv_lens, a.page_table, max_q, max_kv, HQ, HKV, D,
                      D ** -0.5, EPS)


def _bytes(stack):
    return [[x.view(torch.uint8).clone() for x in (L.k_pool, L.v_pool, L.scales)]
            for L in stack.layers[::2]]


def _check(stack, before, t, s):
    cu = pu.cu_of(t)
    for L, (kd, vd, sc) in zip(stack.layers[::2], before):
        rows = L.qkv.reshape(-1, HQ + 2 * HKV, D)
        row = (HQ + 2 * HKV) * D
        xq, xk, xv = L.qkv.split([HQ * D, HKV * D, HKV * D], 1)
        q = torch.empty(rows.shape[0], HQ, D, dtype=torch.bfloat16, device="cuda")
        cache = q8.cache_of(kd, vd, sc, stack.page_table, stack.kv_lens)
        gqa.gqa_packed_rope_append_q8(xq, row, xk, row, xv, row, stack.cu_seqlens, len(t),
                                      rows.shape[0], HQ, HKV, D, L.q_gamma, L.k_gamma, EPS,
                                      L.table, L.table_len, q, None, cache)
        assert pu.status() == 0
        for x, y in ((kd, L.k_pool), (vd, L.v_pool), (sc, L.scales)):
            assert torch.equal(x, y.view(torch.uint8))
        for i, (a, b) in enumerate(zip(t, s)):
            if a == 0:
                continue
            pg, slot = q8.places(stack.page_table, i, PAGE, torch.arange(b, device="cuda"))
            data, byte = q8.quantise(rows[cu[i]:cu[i + 1], HQ + HKV:])
            assert torch.equal(vd[pg, :, slot][b - a:], data)
            assert torch.equal(sc[pg, :, slot, 1][b - a:], byte)
            ro, _, bo, _ = q8.attention64(q[cu[i]:cu[i + 1]], kd[pg, :, slot], sc[pg, :, slot, 0],
                                          vd[pg, :, slot], sc[pg, :, slot, 1], L.window, D ** -0.5)
            pu.check(L.o[cu[i]:cu[i + 1]], ro, bo, f"o of sequence {i}")


@pytest.mark.parametrize("t,s", [([1, 1, 1], [300, 40, 1]), ([4, 2, 3], [300, 40, 3]),
                                 ([130, 1, 0, 70], [200, 300, 7, 70])])
def test_step_over_layers(t, s):
    gu.require_gpu()
    stack = _stack(t, s, (64, 0, 16), 401 + len(t), max(t), 320)
    before = _bytes(stack)
    stack.step()
    assert pu.status() == 0
    _check(stack, before, t, s)


@pytest.mark.parametrize("t", [[1, 1, 1, 1], [2, 1, 30, 4]])
def test_captured_steps_follow_the_lengths(t):
    """A step captured once and replayed while the sequences grow, against eager steps."""
    gu.require_gpu()
    s = [30, 200, 40, 64]
    a = _stack(t, s, (64, 0, 0), 411, max(t), 700)
    b = _stack(t, s, (64, 0, 0), 411, max(t), 700)
    a.step()
    torch.cuda.synchronize()
    graph = a.capture()
    for n in range(3):
        for stack in (a, b):
            stack.kv_lens.copy_(pu.i32([x + 107 * n for x in s]))
            for L in stack.layers:
                L.o.zero_()
        graph.replay()
        b.step()
        torch.cuda.synchronize()
        assert pu.status() == 0
        for L, M in zip(a.layers, b.layers):
            assert torch.equal(L.o, M.o)
            assert torch.equal(L.k_pool.view(torch.uint8), M.k_pool.view(torch.uint8))
