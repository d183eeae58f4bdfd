"""The 8-bit paged attention at the ends of its numbers' ranges: queries and keys of opposite powers
of two, factors that vanish.  By every kernel: a warp per pair (many short caches), up to 8 rows, two
and four groups, the tile kernel."""
import pytest
import torch

import gpu_utils as gu
import packed_utils as pu
from test_gpu_q8 import PagedQ8

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


# tokens, sequences, keys: 8 query heads on 2
KERNELS = [(1, 2, 300), (1, 2, 700), (1, 480, 300), (3, 2, 300), (3, 2, 700), (12, 2, 300),
           (12, 2, 700), (40, 2, 300)]


def _batch(t, n, s, seed, **kw):
    return PagedQ8([t] * n, [s - i % 7 for i in range(n)], 8, 2, 32, seed, **kw)


def _checked(p, *a):
    """A few sequences of each batch."""
    p.run(*a)
    assert pu.status() == 0
    p.check(*a, only=sorted({0, 1, len(p.t) // 2, len(p.t) - 1}))


@pytest.mark.parametrize("t,n,s", KERNELS)
@pytest.mark.parametrize("e", [-118, -100, 100, 110])
def test_queries_and_keys_of_opposite_powers(t, n, s, e):
    """Queries of 2^e, keys of 2^-e: the scores are those of e = 0 (no query below bf16's normal
    numbers)."""
    p = _batch(t, n, s, 950)
    p.q[p.q.abs() < 2.0 ** -7] = 0
    p.q.mul_(2.0 ** e)
    for i in range(n):
        p.rows[i][1].copy_((p.rows[i][1].int() - e).to(torch.uint8))
        p.put(i)
    _checked(p)


@pytest.mark.parametrize("t,n,s", KERNELS)
@pytest.mark.parametrize("window", [0, 50])
def test_rows_of_zeros_under_a_small_scale(t, n, s, window):
    """A row's factor times the call's scale is below 2^-149: visible keys share the weight, hidden
    ones have none."""
    p = _batch(t, n, s, 951)
    p.q[:, 1] = 0
    p.q[:, 6] *= 2.0 ** -120
    _checked(p, window, 2.0 ** -30)
