"""The sources of the 8-bit paged cache without a GPU: the debug build's index checks are there, each
site of a kernel code one kind of access; and the planted caches show the loss of a unit of keys past
the bound in this form, too."""
import os
import re

import pytest
import torch

import packed_utils as pu
import planted_keys
import q8_utils as q8

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "global_causal_gqa_gb300", "csrc")
D = 128


def _text(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name,least", [("paged_stream.cuh", 2), ("paged_q8.cu", 3),
                                        ("paged_q8_few.cu", 2), ("paged_q8_few.cuh", 1),
                                        ("paged_q8_short.cu", 1), ("paged_read.cu", 2)])
def test_sources_with_checks(name, least):
    assert _text(name).count("GQA_IN_BOUNDS(") >= least


def test_sites_are_their_own():
    """Of the streaming kernels (code 8), and of the append and the read-back (code 6)."""
    for names in (("paged_stream.cuh", "paged_decode.cu", "paged_q8.cu", "paged_q8_few.cu",
                   "paged_q8_few.cuh", "paged_q8_short.cu"), ("packed_append.cu", "paged_read.cu")):
        used = {n: {int(x) for x in re.findall(r"kSite \| (\d+)", _text(n))} for n in names}
        for i, a in enumerate(names):
            assert used[a] and max(used[a]) < 1 << 16, a
            for b in names[i + 1:]:
                assert not used[a] & used[b], (a, b)


@pytest.mark.parametrize("S,G", [(50100, 1), (9001, 8)])
def test_every_unit_counts(S, G):
    """As for the bf16 cache: a unit of keys lost, doubled or left out of the value product alone
    moves the output past the bound."""
    gen = torch.Generator().manual_seed(S + G)
    q = planted_keys.queries(gen, 1, G, D, "cpu")
    k, v = (torch.randn(S, 1, D, generator=gen).double() for _ in range(2))
    at, head, dim = planted_keys.plant(q, k, v)
    rows = [*q8.quantise(k), *q8.quantise(v)]
    k, v = q8.values(*rows[:2]), q8.values(*rows[2:])
    o, _, bound, _ = q8.attention64(q, *rows, 0, D ** -0.5)
    n = len(at)
    for u in sorted({0, 1, n // 3, n // 2, n - 2, n - 1}):
        unit, h = slice(u * planted_keys.UNIT, (u + 1) * planted_keys.UNIT), int(head[u])
        x = (k[:, 0] @ q[0, h].double()) * D ** -0.5
        for lost, values in ((0.0, 0.0), (2.0, 2.0), (1.0, 0.0), (1.0, 2.0)):
            p = torch.exp(x - x.max())
            p[unit] *= lost
            p /= p.sum()
            if lost == 1.0:
                p[unit] *= values
            worst = ((p @ v[:, 0] - o[0, h]).abs() / bound[0, h]).max()
            assert worst > 2, (u, lost, values, float(worst))


def test_the_plain_form_of_the_numbers():
    """quantise and values against the definition, element by element."""
    gen = torch.Generator().manual_seed(9)
    x = torch.randn(50, D, generator=gen).double() * torch.exp2(
        torch.randint(-40, 40, (50, 1), generator=gen).double())
    x[3] = 0
    data, byte = q8.quantise(x)
    grid = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    grid = grid[torch.isfinite(grid)]
    for r in range(50):
        e = int(byte[r]) - 127
        most = float(x[r].abs().max())
        assert most <= 448 * 2.0 ** e and (most > 448 * 2.0 ** (e - 1) or e == q8.E_LO)
        y = x[r] / 2.0 ** e
        nearest = (y[:, None] - grid[None]).abs().amin(1)
        assert torch.equal((q8.numbers(data[r]) - y).abs(), nearest)
    assert torch.equal(q8.values(data, byte)[3], torch.zeros(D, dtype=torch.float64))
