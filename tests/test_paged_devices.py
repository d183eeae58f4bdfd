"""The paged cache and PagedStack without a GPU: tensors on different devices, and offsets with
a stride, would give the kernels addresses of something else, and are refused."""
import dataclasses

import pytest
import torch

import global_causal_gqa_gb300 as gqa
from test_paged_stack_args import _layer, _stack


@pytest.mark.parametrize("which", range(4))
def test_a_cache_lies_on_one_device(which):
    k = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    ts = [k, k.clone(), torch.zeros(3, 5, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)]
    gqa.make_paged_kv(*ts)
    ts[which] = ts[which].to("meta")
    with pytest.raises(ValueError, match="one device"):
        gqa.make_paged_kv(*ts)


@pytest.mark.parametrize("field", ["qkv", "o", "q_gamma", "k_gamma", "table"])
def test_a_stack_lies_on_one_device(field):
    L = _layer()
    with pytest.raises(ValueError, match="one device"):
        _stack([_layer(), dataclasses.replace(L, **{field: getattr(L, field).to("meta")})])


def test_offsets_of_a_stack():
    wide = torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="cu_seqlens"):
        _stack([_layer()], wide[:, 0])
    with pytest.raises(ValueError, match="one device"):
        _stack([_layer()], torch.zeros(3, dtype=torch.int32, device="meta"))
    _stack([_layer()], wide[:, 0].contiguous())
