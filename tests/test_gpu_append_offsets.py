"""Offsets that contradict one another, in the append: the sequences with sound ones are written,
rows that belong to none stay as they were, and the status word tells of every one that does
not hold, wherever it stands in the batch and whether or not a row falls to it."""
import pytest
import torch

import global_causal_gqa_gb300 as gqa
import gpu_utils as gu
import packed_utils as pu
from test_gpu_packed import _gen, _randn, _table
from test_gpu_packed_offsets import BAD, _claims

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


def _append(cu, total, d=64):
    """q and what a call with offsets cu made of it and of k."""
    n = len(cu) - 1
    q, k, v = (_randn(_gen(430 + i), total, d) for i in range(3))
    tab = _table(d, 4096)
    qo = torch.full((total, 1, d), 3.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((total, 1, d), 3.0, dtype=torch.bfloat16, device="cuda")
    gqa.gqa_packed_rope_append(q, d, k, d, v, d, pu.i32(cu), n, total, 1, 1, d, None, None, 0.0, tab,
                               4096, qo, ko, None)
    return q, qo, ko


def _check_rows(x, y, cu, total):
    sound, n = _claims(cu, total)
    # rows over which the offsets decrease may go to any sequence that claims them, or to none
    loose = [any(b <= r < a for a, b in zip(cu, cu[1:])) for r in range(total)]
    for i, a, b in sound:
        at = torch.tensor([r for r in range(a, b) if not loose[r]], dtype=torch.long, device="cuda")
        if len(at) == 0:
            continue
        want = pu.rope64(x[at][:, None], at - a, 1e4)
        h = want.abs()
        half = h.shape[-1] // 2
        pair = torch.cat([h[..., :half] + h[..., half:]] * 2, -1)
        # one rounding to bf16; the table's and the two products' fp32 roundings: 8 of a pair's
        # length
        pu.check(y[at], want, pu.BF16 * h + 16 * pu.FP32 * 1.5 * pair, f"rows of sequence {i}")
    none = torch.tensor([c == 0 for c in n], device="cuda")
    assert (y[none] == 3).all()


@pytest.mark.parametrize("cu", BAD)
def test_append(cu):
    q, qo, _ = _append(cu, 10)
    assert pu.status() == -1
    _check_rows(q, qo, cu, 10)


@pytest.mark.parametrize("total", [64, 608, 609, 2000])
@pytest.mark.parametrize("behind", [1, 40, 700])
def test_append_behind_many_sound_ones(total, behind):
    """A few tokens and many: both forms of the kernel."""
    cu = list(range(0, total + 1, 8))
    cu += [total] * (cu[-1] != total) + [total + 3 * (i + 1) for i in range(behind)]
    q, qo, ko = _append(cu, total)
    assert pu.status() == -1
    _check_rows(q, qo, cu, total)


@pytest.mark.parametrize("total", [5, 700])
def test_append_first_sequence_ends_at_row_0(total):
    q, qo, ko = _append([-3, 0, total], total)
    assert pu.status() == -1
    _check_rows(q, qo, [-3, 0, total], total)


@pytest.mark.parametrize("total", [5, 700])
def test_sound_offsets_leave_the_status_alone(total):
    """Empty sequences anywhere, among them behind the last row."""
    cu = [0, 0, 2, 2, 2, total, total, total]
    q, qo, ko = _append(cu, total)
    assert pu.status() == 0
    _check_rows(q, qo, cu, total)
