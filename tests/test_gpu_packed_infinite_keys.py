"""Keys with a negative infinite element that every query meets with a positive one: their scores
are -inf and their weights 0.  A row that sees other keys attends to those alone; a row that sees
no other has softmax 0 / 0, NaN, and lse -inf, whichever kernel computes it and however its keys
are split."""
import math

import pytest
import torch

import global_causal_gqa_gb300 as gqa
import gpu_utils as gu
import packed_utils as pu
from test_gpu_packed import D, Paged, _packed

pytestmark = pytest.mark.gpu
AT = 5    # the element


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (6, 2), (2, 2)])
@pytest.mark.parametrize("n,first", [(20, 3), (300, 1), (300, 150), (300, 300)])
def test_packed(Hq, Hkv, n, first):
    def edit(q, k, v, cu):
        q[:, AT::D] = 1.0
        k[:first, AT::D] = -math.inf
    q, k, v, cu, o, L, scale = _packed([n, 40], Hq, Hkv, 0, 401, edit=edit)
    assert torch.isnan(o[:first]).all() and (L[:, :first] == -math.inf).all()
    for a, b in ((first, n), (n, n + 40)):
        if a < b:
            ro, rl, bo, bl = pu.attention64(q[a:b], k[a:b], v[a:b], 0, scale)
            pu.check(o[a:b], ro, bo, "rows that see other keys")
            pu.check(L[:, a:b], rl, bl, "their lse")


def _paged(t, s, Hq, Hkv, infinite, max_kv=None):
    p = Paged(t, s, Hq, Hkv, 16, 410 + sum(t), max_kv=max_kv)
    p.q[:, :, AT] = 1.0
    for i, n in enumerate(infinite):
        p.k[i][:n, :, AT] = -math.inf
        pu.put(p.kp, p.table, i, p.k[i])
    p.run()
    assert pu.status() == 0
    return p


# decode by whole pairs, decode and drafts in chunks, tiles whole, tiles in spans
SHAPES = [([1, 1], [137, 60], 8, 2), ([1, 1], [9001, 700], 8, 2), ([2, 2], [9001, 700], 8, 1),
          ([40, 3], [200, 60], 8, 2), ([40, 3], [9001, 700], 8, 1)]


@pytest.mark.parametrize("t,s,Hq,Hkv", SHAPES)
def test_paged_all_keys(t, s, Hq, Hkv):
    p = _paged(t, s, Hq, Hkv, [s[0], 0])
    o, n = p.out(), t[0]
    assert torch.isnan(o[:n]).all() and (p.L[:, :n] == -math.inf).all()
    ro, rl, bo, bl = pu.attention64(p.q[n:], p.k[1], p.v[1], 0, D ** -0.5)
    pu.check(o[n:], ro, bo, "the other sequence")
    pu.check(p.L[:, n:], rl, bl, "its lse")


@pytest.mark.parametrize("t,s,Hq,Hkv", SHAPES)
def test_paged_some_keys(t, s, Hq, Hkv):
    """Whole chunks and spans without a weight, among others with."""
    cut = [(a - b) // 2 for a, b in zip(s, t)]
    p = _paged(t, s, Hq, Hkv, cut)
    o = p.out()
    for i, c in enumerate(cut):
        a, b = p.cu[i], p.cu[i + 1]
        ro, rl, bo, bl = pu.attention64(p.q[a:b], p.k[i][c:], p.v[i][c:], 0, D ** -0.5)
        pu.check(o[a:b], ro, bo, f"o of sequence {i}")
        pu.check(p.L[:, a:b], rl, bl, f"lse of sequence {i}")


def test_the_workspace_tells_the_shapes_apart():
    """The shapes above do run split and whole."""
    def size(t, s, Hq, Hkv):
        return gqa.gqa_attn_paged_workspace_bytes(2, sum(t), max(t), max(s), Hq, Hkv, D)
    assert [size(*x) > 0 for x in SHAPES] == [False, True, True, False, True]
