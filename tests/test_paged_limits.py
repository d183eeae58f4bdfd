"""The documented limits on what a packed or paged call counts, without a GPU: the workspace query
answers 0 and the call refuses, both at the same bound."""
import numpy as np
import pytest

import global_causal_gqa_gb300 as gqa

P = 0x10000   # an aligned address that no call here dereferences
M = 2 ** 31 - 1


def _call(nseq, total, max_q, max_kv, Hq, Hkv):
    a = np.zeros(1, dtype=gqa.PAGED_KV_DTYPE)
    for n, x in dict(k=P, v=P, page_table=P, kv_lens=P, num_pages=4, Hkv=Hkv, page_size=16, d=128,
                     max_pages=1 << 26).items():
        a[n] = x
    # a workspace of one byte: a shape that is not refused stops there, or needs none
    return gqa.gqa_attn_paged(P, Hq * 128, a, P, nseq, total, max_q, max_kv, Hq, 0, 1.0, 2 * P,
                              Hq * 128, P, P, 1, stream=1, check=False)


def _size(*a):
    return gqa.gqa_attn_paged_workspace_bytes(*a, 128)


# nseq, total, max_q, max_kv, Hq, Hkv
FITS = [(15, 15, 1, 2 ** 30, 64, 8),                  # 15 * 8 * 2^24 units
        (127, 127, 1, 2 ** 30, 1, 1),
        (M // 1024 - 1, 2 ** 20, 1, 65536, 1, 1),
        (2, 2 ** 30, 2 ** 30, 2 ** 30, 1, 1),
        (4, 64, 64, 2 ** 30, 8, 8)]
PASS = [(17, 17, 1, 2 ** 30, 64, 8),
        (128, 128, 1, 2 ** 30, 1, 1),
        (M // 1024 + 1, 2 ** 20, 1, 65536, 1, 1),
        (M, 2 ** 30, 1, 2 ** 30, 2 ** 24, 2 ** 24),   # past 64 bits as well
        (2, 2 ** 30 + 1, 17, 64, 8, 8), (2, M, 1, 64, 8, 8), (2, M, 40, 64, 8, 8),
        (2 ** 30, 2 ** 30, 17, 64, 8, 8), (M, 2 ** 30, 40, 2 ** 30, 2 ** 24, 2 ** 24)]


@pytest.mark.parametrize("shape", FITS)
def test_up_to_the_limits(shape):
    assert _size(*shape) > 0
    assert _call(*shape) == -7            # the workspace is too small for it


@pytest.mark.parametrize("shape", PASS)
def test_beyond_them(shape):
    assert _size(*shape) == 0
    assert _call(*shape) == -2


def test_packed_prompts():
    def call(nseq, total, Hkv):
        row = Hkv * 128
        return gqa.gqa_attn_packed(P, row, P, row, P, row, 2 * P, row, P, P, nseq, total, Hkv, Hkv,
                                   128, 0, 1.0, stream=1, check=False)
    assert call(2 ** 28, 2 ** 28, 8) == -2
    assert call(M, 2 ** 30, 2 ** 24) == -2


@pytest.mark.parametrize("total", [M - 511, M - 63, M])
def test_append_rows(total):
    assert gqa.gqa_packed_rope_append(None, 0, P, 64, None, 0, P, 2, total, 0, 1, 64, None, None, 0.0,
                                      P, 64, None, 2 * P, None, stream=1, check=False) == -2
