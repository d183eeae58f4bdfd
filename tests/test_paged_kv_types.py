"""make_paged_kv without a GPU: tensors whose elements have the right size but another type would
be read as something else, and are refused."""
import pytest
import torch

import global_causal_gqa_gb300 as gqa


def _tensors(pool=torch.bfloat16, table=torch.int32, lens=torch.int32):
    k = torch.zeros(4, 2, 16, 128, dtype=pool)
    return [k, k.clone(), torch.zeros(3, 5, dtype=table), torch.zeros(3, dtype=lens)]


def test_the_types_that_fit():
    assert int(gqa.make_paged_kv(*_tensors())["num_pages"][0]) == 4


@pytest.mark.parametrize("pool", [torch.float16, torch.int16, torch.uint8, torch.float32])
def test_pools_of_another_type(pool):
    with pytest.raises(ValueError, match="bfloat16"):
        gqa.make_paged_kv(*_tensors(pool=pool))
    one = _tensors()
    one[1] = one[1].to(pool)
    with pytest.raises(ValueError, match="bfloat16"):
        gqa.make_paged_kv(*one)


@pytest.mark.parametrize("kind", [torch.float32, torch.int64, torch.int16])
@pytest.mark.parametrize("which", ["table", "lens"])
def test_tables_and_lengths_of_another_type(kind, which):
    with pytest.raises(ValueError, match="int32"):
        gqa.make_paged_kv(*_tensors(**{which: kind}))
