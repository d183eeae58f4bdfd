"""Offsets and lengths that contradict one another: the sequences with sound ones are computed,
rows that belong to none stay as they were, and the status word tells of every one that does
not hold, wherever it stands in the batch and whether or not a row falls to it."""
import pytest
import torch

import global_causal_gqa_gb300 as gqa
import gpu_utils as gu
import packed_utils as pu
from test_gpu_packed import D, _gen, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


def _claims(cu, total):
    """(sequence, first row, end) of the sound sequences, and how many of them claim each row."""
    sound = [(i, a, b) for i, (a, b) in enumerate(zip(cu, cu[1:])) if 0 <= a <= b <= total]
    n = [sum(a <= r < b for _, a, b in sound) for r in range(total)]
    return sound, n


BAD = [[0, 5, 3, 9], [-1, 4, 6, 9], [0, 4, 6, 13], [0, 10, 30], [-5, 0, 10], [0, 10, 5],
       [0, 4, 10, 11], [0, 9, 2 ** 31 - 1], [-2 ** 31, 3, 10]]


@pytest.mark.parametrize("cu", BAD)
@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (2, 2), (16, 1)])
def test_packed_attention(cu, Hq, Hkv):
    total = 10
    qkv = _randn(_gen(421), total, (Hq + 2 * Hkv) * D)
    row = qkv.shape[1]
    q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], 1)
    o = torch.full((total, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    L = torch.full((Hq, total), 3.0, device="cuda")
    gqa.gqa_attn_packed(q, row, k, row, v, row, o, Hq * D, L, pu.i32(cu), len(cu) - 1, total, Hq,
                        Hkv, D, 0, D ** -0.5)
    assert pu.status() == -1
    sound, n = _claims(cu, total)
    for i, a, b in sound:
        rows = [r for r in range(a, b) if n[r] == 1]
        if not rows:
            continue
        at = torch.tensor(rows, device="cuda")
        ro, rl, bo, bl = pu.attention64(q[a:b].reshape(-1, Hq, D), k[a:b].reshape(-1, Hkv, D),
                                        v[a:b].reshape(-1, Hkv, D), 0, D ** -0.5)
        pu.check(o[at], ro[at - a], bo[at - a], f"o of sequence {i}")
        pu.check(L[:, at], rl[:, at - a], bl[:, at - a], f"lse of sequence {i}")
    for r in range(total):
        if n[r] == 0:
            assert (o[r] == 3).all() and (L[:, r] == 3).all()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (16, 2)])
@pytest.mark.parametrize("behind", [1, 36, 70])
def test_packed_attention_behind_many_sound_ones(Hq, Hkv, behind):
    """Single tokens fill every row; the sequences behind them pass the end."""
    good = 64
    cu = list(range(good + 1)) + [good + 6 * (i + 1) for i in range(behind)]
    q, k = _randn(_gen(422), good, Hq * D), _randn(_gen(423), good, Hkv * D)
    v = _randn(_gen(424), good, Hkv * D)
    o = torch.full((good, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    gqa.gqa_attn_packed(q, Hq * D, k, Hkv * D, v, Hkv * D, o, Hq * D, None, pu.i32(cu), len(cu) - 1,
                        good, Hq, Hkv, D, 0, 1.0)
    assert pu.status() == -1
    # a single key has weight 1
    want = v.reshape(good, Hkv, D).repeat_interleave(Hq // Hkv, 1)
    assert torch.equal(o, want)
