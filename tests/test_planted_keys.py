"""The planted caches of the GPU tests, on the CPU: a unit of keys that a computation loses, counts
twice, or leaves out of the value product alone moves the output past the error bound."""
import pytest
import torch

import packed_utils as pu
import planted_keys

D = 128


def _attend(q, k, v, keep, values):
    """One query in 64 bits with every key's weight times `keep`, its value's times `values`."""
    x = (k.double() @ q.double()) * D ** -0.5
    p = torch.exp(x - x.max()) * keep
    return (p / p.sum() * values) @ v.double()


@pytest.mark.parametrize("S,G", [(50100, 1), (50100, 8), (9001, 4), (9001, 8), (400000, 2)])
def test_every_unit_counts(S, G):
    gen = torch.Generator().manual_seed(S + G)
    q = planted_keys.queries(gen, 1, G, D, "cpu")
    k, v = (torch.randn(S, 1, D, generator=gen).to(torch.bfloat16) for _ in range(2))
    at, head, dim = planted_keys.plant(q, k, v)
    o, _, bound, _ = pu.attention64(q, k, v, 0, D ** -0.5)
    one = torch.ones(S, dtype=torch.float64)
    n = len(at)
    for u in sorted({0, 1, n // 3, n // 2, n - 2, n - 1}):
        unit = slice(u * planted_keys.UNIT, (u + 1) * planted_keys.UNIT)
        h = int(head[u])
        for lost, values in ((0.0, 0.0), (2.0, 2.0), (1.0, 0.0), (1.0, 2.0)):
            keep, val = one.clone(), one.clone()
            keep[unit] = lost
            val[unit] = values if lost == 1.0 else 1.0
            bad = _attend(q[0, h], k[:, 0], v[:, 0], keep, val)
            worst = ((bad - o[0, h]).abs() / bound[0, h]).max()
            assert worst > 2, (u, lost, values, float(worst))


def test_the_planted_keys_have_the_weight():
    gen = torch.Generator().manual_seed(5)
    q = planted_keys.queries(gen, 3, 8, D, "cpu")
    k, v = (torch.randn(20000, 2, D, generator=gen).to(torch.bfloat16) for _ in range(2))
    at, head, dim = planted_keys.plant(q, k, v)
    for h in range(8):
        x = (k[:, h // 4].double() @ q[2, h].double()) * D ** -0.5
        p = torch.softmax(x, 0)
        mine = at[head == h % 4]
        assert p[mine].sum() > 0.999
        assert p[mine].max() < 1.01 * p[mine].min()
