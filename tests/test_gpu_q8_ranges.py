"""The 8-bit paged attention at the ends of its numbers' ranges: queries and keys of opposite powers
of two, factors that vanish, scores far from zero, values of tiny powers.  By every kernel: a warp
per pair (many short caches), up to 8 rows, two and four groups, the tile kernel."""
import math

import pytest
import torch

import gpu_utils as gu
import packed_utils as pu
import q8_utils as q8
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


@pytest.mark.parametrize("t,n,s", KERNELS)
@pytest.mark.parametrize("up", [-60, 0, 60])
@pytest.mark.parametrize("far", [20, 30])
def test_scores_far_from_zero(t, n, s, up, far):
    """Scores of 2^(far + 3): 2^12 or 2^18 in every element of queries and keys, some keys half of
    it, scale 1/16 and 128 dims.  All products and sums are powers of two, so a row's weights are
    exact: the same for the keys that it sees of the larger ones, none for the others (2^(far + 2)
    below), and the result is the mean of their values.  Weights times the values' powers of two
    are powers of two in the kernels' 8-bit columns or f16, and their products with 4-bit numbers
    exact; what is left is fp32 sums (of n terms: n 2^-24 of their magnitudes, twice that where a
    tensor core truncates), at most 16 factors, each off by 2^-22, that take the result from one
    reference to another, and one rounding to bf16.  lse: six roundings to fp32 of the score, 2^-24
    each (the scale times log2 e, the factors, the score, ln 2, the product with it, the sum)."""
    a = far // 2 + 2
    p = _batch(t, n, s, 952, spread=6)
    p.q.fill_(2.0 ** a)
    some = sorted({0, 1, n // 2, n - 1})
    for i in range(n):
        x = torch.full((p.s[i], 2, 128), 2.0 ** (far - a), dtype=torch.float64, device="cuda")
        x[1::3] /= 2
        p.rows[i][0], p.rows[i][1] = q8.quantise(x)
        p.rows[i][3] = (p.rows[i][3].int() + up).to(torch.uint8)
        p.put(i)
    p.run(0, 1 / 16)
    assert pu.status() == 0
    for i in some:
        v = q8.values(p.rows[i][2], p.rows[i][3])
        on = torch.arange(p.s[i], device="cuda") % 3 != 1
        for r in range(t):
            see = on & (torch.arange(p.s[i], device="cuda") <= p.s[i] - t + r)
            m = int(see.sum())
            mean = v[see].mean(0).repeat_interleave(4, 0)
            off = (2 * p.s[i] * pu.FP32 + 2.0 ** -18) * v[see].abs().mean(0).repeat_interleave(4, 0)
            bound = off + pu.BF16 * (mean.abs() + off)
            pu.check(p.out()[p.cu[i] + r], mean, bound, f"row {r} of sequence {i}")
            z = 2.0 ** (far + 3) + math.log(m)
            pu.check(p.L[:, p.cu[i] + r], torch.full((8,), z, dtype=torch.float64, device="cuda"),
                     torch.full((8,), z * 2.0 ** -21, dtype=torch.float64, device="cuda"), "lse")


@pytest.mark.parametrize("t,n,s", KERNELS[:-1])
def test_values_of_tiny_powers(t, n, s):
    """Values of the format's last two powers of two: what is lost of a weight is relative to them,
    not to a larger value that is not there.  (Not by the tile kernel, to which many of them are
    below bf16's normal numbers.)"""
    p = _batch(t, n, s, 953, spread=3)
    for i in range(n):
        p.rows[i][3] = (p.rows[i][3].int() - 118).clamp_min(1).to(torch.uint8)
        p.put(i)
    _checked(p)
