"""What the tensor maps of the library span, worked out from the sources (no GPU needed).

The encoder's description asks for strides that are multiples of the ones before.  Some maps here
take the halves of a row as a dimension, or rows of the caller's own stride, and are outside of it;
each is named below.  What every map keeps to instead is its tensor: the elements that its dimensions
and strides reach are the tensor's own, the last one of them its last, so that no address between
them belongs to anything else."""
import os
import re
from types import SimpleNamespace

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "global_causal_gqa_gb300", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _value(expr, env):
    expr = re.sub(r"\((cu)?uint(32|64)_t\)", "", expr).replace("/", "//")
    return eval(expr, {"__builtins__": {}}, env)          # of the repository's own sources


def _arrays(text):
    """Every `name[n] = {...}` in the text: (name, place, expressions)."""
    return [(m.group(1), m.start(), [x.strip() for x in re.split(r",(?![^()]*\))", m.group(2))])
            for m in re.finditer(r"\b(\w+)\[\d\] = \{([^}]*)\}", text)]


def _maps():
    """(file, what is mapped, element bytes, dims, strides) of every map, as expressions."""
    out = []
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        text = _code(name)
        arrays = _arrays(text)

        def last(array, at):
            found = [a for a in arrays if a[0] == array and a[1] < at]
            assert found, (name, array)
            return found[-1][2]
        for m in re.finditer(r"make_(bf16|byte)_map\(\s*&?\w+,\s*([^,]+),\s*(\d),\s*(\w+),\s*(\w+),",
                             text):
            dims, strides = last(m.group(4), m.start()), last(m.group(5), m.start())
            assert len(dims) == int(m.group(3)) == len(strides) + 1
            out.append((name, m.group(2), 2 if m.group(1) == "bf16" else 1, dims, strides))
        for m in re.finditer(r"return fn\(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,", text):
            out.append((name, "base", 2, last("dims", m.start()), last("strides", m.start())))
    return out


# sizes of a call: pools, rows of a fused projection and of the tests' own strides, heads
SIZES = [dict(pages=pages, hkv=hkv, page=page, total=total, hq=hq, pad=pad)
         for pages, hkv, page in ((1, 1, 16), (7, 3, 32), (900, 8, 64), (5, 2, 128))
         for total, hq, pad in ((1, 1, 0), (37, 8, 8), (4000, 64, 2048))]


def _env(z):
    c = SimpleNamespace(num_pages=z["pages"], Hkv=z["hkv"], page_size=z["page"])
    row = 128 * (z["hq"] + z["pad"] // 8 * 2)
    a = SimpleNamespace(total=z["total"], Hq=z["hq"], Hkv=z["hkv"], q_stride=z["hq"] * 128 + z["pad"],
                        o_stride=z["hq"] * 128 + 8, k_stride=row + z["hkv"] * 128,
                        v_stride=z["hkv"] * 128 + 8)
    return dict(c=c, a=a, page=z["page"], kD=128, d=512, rows=z["total"], slabs=z["hq"])


def _bytes(what, size, e):
    """The bytes from a tensor's first element to its last."""
    a, c = e["a"], e["c"]
    rows = {"a.q": (a.q_stride, a.Hq), "a.o": (a.o_stride, a.Hq), "a.k": (a.k_stride, a.Hkv),
            "a.v": (a.v_stride, a.Hkv)}
    if what in rows:
        stride, heads = rows[what]
        return ((a.total - 1) * stride + heads * 128) * size
    return c.num_pages * c.Hkv * c.page_size * 128 * size


def test_every_map_is_found():
    text = "".join(_code(n) for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh")))
    made = len(re.findall(r"(?<!bool )\bmake_(?:bf16|byte)_map\(", text))
    assert made == 10 and len(_maps()) == made + 4


@pytest.mark.parametrize("z", range(len(SIZES)))
def test_maps_span_their_tensors_alone(z):
    e = _env(SIZES[z])
    for name, what, size, dims, strides in _maps():
        kd = dict(e, d=512 if "kD" not in dims[0] else 128)
        n, s = [_value(x, kd) for x in dims], [_value(x, kd) for x in strides]
        assert all(x % 16 == 0 and 0 < x < 1 << 40 for x in s), (name, what)
        reach = n[0] * size + sum((k - 1) * x for k, x in zip(n[1:], s))
        if what == "base":
            assert reach == n[0] * e["rows"] * e["slabs"] * size, (name, what)
        else:
            assert reach == _bytes(what, size, e), (name, what)


def test_the_maps_whose_strides_are_not_multiples():
    """The only ones: pages as rows of two halves, packed keys and values likewise, and rows of any
    stride that the call allows."""
    odd = set()
    for z in SIZES:
        e = _env(z)
        for name, what, size, dims, strides in _maps():
            s = [_value(x, e) for x in strides]
            if any(y % x for x, y in zip(s, s[1:])):
                odd.add((name, what))
    assert odd == {("packed_prefill.cu", x) for x in ("a.q", "a.o", "a.k", "a.v", "c.k", "c.v")} | \
        {("paged_decode.cu", x) for x in ("c.k", "c.v")}


def test_one_map_over_two_pools_would_span_what_lies_between():
    """The form that the 8-bit kernels had before: the pools' distance as a dimension's stride."""
    page, pages, apart = 16, 10, 12 << 30
    n, s = [128, 8, 2, page // 8, pages], [128, apart, 8 * 128, page * 128]
    reach = n[0] + sum((k - 1) * x for k, x in zip(n[1:], s))
    assert reach == apart + pages * page * 128 and apart > 1000 * pages * page * 128
