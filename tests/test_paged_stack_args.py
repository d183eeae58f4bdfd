"""PagedStack and the paged calls without a GPU: tensors that do not fit one another are refused
when the stack is built, and a bound on the keys that 32 bits do not cover by the call."""
import dataclasses

import numpy as np
import pytest
import torch

import global_causal_gqa_gb300 as gqa
from global_causal_gqa_gb300.model_step import PagedLayer, PagedStack

D, HQ, HKV = 128, 4, 2


def _layer(total=6):
    pool = torch.zeros(8, HKV, 16, D, dtype=torch.bfloat16)
    return PagedLayer(pool, pool.clone(), torch.zeros(total, (HQ + 2 * HKV) * D, dtype=torch.bfloat16),
                      torch.zeros(total, HQ, D, dtype=torch.bfloat16), torch.ones(D), torch.ones(D),
                      torch.zeros(32 * D), 32, 0)


def _stack(layers, cu=None):
    return PagedStack(layers, torch.zeros(3, dtype=torch.int32) if cu is None else cu,
                      torch.zeros(2, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32), 3, 32,
                      HQ, HKV, D, D ** -0.5)


def test_a_stack_that_fits():
    s = _stack([_layer(), _layer()])
    assert s.total == 6 and s.nseq == 2 and s.q.shape == (6, HQ, D) and len(s.caches) == 2


@pytest.mark.parametrize("field,value", [
    ("qkv", torch.zeros(5, (HQ + 2 * HKV) * D, dtype=torch.bfloat16)),
    ("qkv", torch.zeros(6, (HQ + 2 * HKV) * D)),
    ("qkv", torch.zeros(6, 2 * (HQ + 2 * HKV) * D, dtype=torch.bfloat16)[:, ::2]),
    ("o", torch.zeros(6, HQ + 1, D, dtype=torch.bfloat16)),
    ("o", torch.zeros(5, HQ, D, dtype=torch.bfloat16)),
    ("k_pool", torch.zeros(8, HKV, 32, D, dtype=torch.bfloat16)),
    ("q_gamma", torch.ones(D - 1)), ("k_gamma", torch.ones(D, dtype=torch.bfloat16)),
    ("table", torch.zeros(31 * D)),
])
def test_layers_that_do_not_fit(field, value):
    with pytest.raises(ValueError):
        _stack([_layer(), dataclasses.replace(_layer(), **{field: value})])


def test_other_heads_and_offsets():
    pool = torch.zeros(8, HKV + 1, 16, D, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        _stack([dataclasses.replace(_layer(), k_pool=pool, v_pool=pool.clone())])
    for cu in (torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)):
        with pytest.raises(ValueError):
            _stack([_layer()], cu)


def test_keys_beyond_the_bound():
    P = 0x10000   # an aligned address that is not dereferenced
    a = np.zeros(1, dtype=gqa.PAGED_KV_DTYPE)
    for n, x in dict(k=P, v=P, page_table=P, kv_lens=P, num_pages=4, Hkv=2, page_size=16, d=128,
                     max_pages=1 << 28).items():
        a[n] = x
    for max_q in (1, 64):
        for max_kv in (2 ** 30 + 1, 2 ** 31 - 1):
            assert gqa.gqa_attn_paged_workspace_bytes(2, 64, max_q, max_kv, 8, 2, 128) == 0
            assert gqa.gqa_attn_paged(P, 1024, a, P, 2, 64, max_q, max_kv, 8, 0, 1.0, 2 * P, 1024, P,
                                      P, 1 << 40, stream=1, check=False) == -2
    assert gqa.gqa_attn_packed(P, 1024, P, 256, P, 256, 2 * P, 1024, P, P, 2, 2 ** 30 + 1, 8, 2, 128,
                               0, 1.0, stream=1, check=False) == -2
