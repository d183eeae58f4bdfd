"""The 8-bit paged cache without a GPU: wrong arguments are refused on the host before anything
is launched, workspace sizes follow from the shape, and the binding checks its tensors."""
import dataclasses

import numpy as np
import pytest
import torch

import global_causal_gqa_gb300 as gqa
from test_paged_stack_args import D, HKV, _layer, _stack

P = 0x10000   # an aligned address that no call here dereferences
NAN, INF = float("nan"), float("inf")


def _cache(**kw):
    a = np.zeros(1, dtype=gqa.PAGED_KV_Q8_DTYPE)
    f = dict(k=P, v=P, scales=P, page_table=P, kv_lens=P, num_pages=4, Hkv=2, page_size=16, d=128,
             max_pages=2, reserved=0)
    f.update(kw)
    for n, x in f.items():
        a[n] = x
    return a


def _append(**kw):
    a = dict(q=P, q_stride=1024, k=P, k_stride=256, v=P, v_stride=256, cu_seqlens=P, nseq=2,
             total=10, Hq=8, Hkv=2, d=128, q_gamma=P, k_gamma=P, eps=1e-6, table=P, table_len=64,
             q_out=2 * P, k_out=3 * P, cache=_cache())
    a.update(kw)
    return gqa.gqa_packed_rope_append_q8(*a.values(), stream=1, check=False)


def _paged(**kw):
    a = dict(q=P, q_stride=1024, cache=_cache(), cu_seqlens=P, nseq=2, total=10, max_q=5,
             max_kv=32, Hq=8, window=0, scale=1.0, o=2 * P, o_stride=1024, lse=P, workspace=P,
             workspace_bytes=1 << 50)
    a.update(kw)
    return gqa.gqa_attn_paged_q8(*a.values(), stream=1, check=False)


def _read(**kw):
    a = dict(cache=_cache(), cu_seqlens=P, nseq=2, total=10, k_out=2 * P, k_stride=256, v_out=3 * P,
             v_stride=256)
    a.update(kw)
    return gqa.gqa_paged_read_q8(*a.values(), stream=1, check=False)


BAD_CACHES = [
    (_cache(k=0), -1), (_cache(v=0), -1), (_cache(scales=0), -1), (_cache(kv_lens=0), -1),
    (_cache(page_table=0), -1), (_cache(num_pages=0), -1), (_cache(max_pages=0), -1),
    (_cache(reserved=1), -1), (_cache(Hkv=0), -1), (_cache(page_size=24), -2),
    (_cache(page_size=256), -2), (_cache(num_pages=1 << 30, Hkv=2), -2), (_cache(v=P + 8), -3),
    (_cache(scales=P + 8), -3), (_cache(page_table=P + 2), -3), (_cache(kv_lens=P + 1), -3)]


@pytest.mark.parametrize("cache,code", BAD_CACHES)
def test_caches_refused(cache, code):
    assert _append(cache=cache) == code
    assert _paged(cache=cache) == code
    assert _read(cache=cache) == code


@pytest.mark.parametrize("kw,code", [
    (dict(cache=None), -1), (dict(k=0), -1), (dict(q=0), -1), (dict(q_out=0), -1), (dict(v=0), -1),
    (dict(table=0), -1), (dict(cu_seqlens=0), -1), (dict(nseq=0), -1), (dict(total=0), -1),
    (dict(Hq=0), -1), (dict(Hkv=0), -1), (dict(table_len=0), -1), (dict(eps=-1.0), -1),
    (dict(eps=NAN), -1), (dict(eps=INF), -1), (dict(d=96), -2), (dict(total=2 ** 31 - 1), -2),
    (dict(q_stride=1020), -1), (dict(k_stride=128), -1), (dict(v_stride=0), -1),
    (dict(q_out=P, q_stride=1032), -1), (dict(k_out=P, k_stride=264), -1), (dict(q=P + 4), -3),
    (dict(k_out=P + 4), -3), (dict(q_gamma=P + 4), -3), (dict(table=P + 8), -3),
    (dict(v=P + 2), -3), (dict(cu_seqlens=P + 2), -3), (dict(cache=_cache(Hkv=1)), -1),
    (dict(cache=_cache(d=64)), -1)])
def test_append_refusals(kw, code):
    assert _append(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), -1), (dict(cache=None), -1), (dict(o=0), -1), (dict(cu_seqlens=0), -1),
    (dict(nseq=0), -1), (dict(total=0), -1), (dict(max_q=0), -1), (dict(max_kv=4), -1),
    (dict(Hq=0), -1), (dict(Hq=7), -1), (dict(scale=0.0), -1), (dict(scale=NAN), -1),
    (dict(scale=INF), -1), (dict(cache=_cache(d=256), q_stride=2048, o_stride=2048), -2),
    (dict(Hq=130, q_stride=130 * 128, o_stride=130 * 128), -2),
    (dict(max_kv=2 ** 30 + 1), -2), (dict(total=2 ** 30 + 1), -2),
    (dict(q_stride=1022), -1), (dict(o_stride=512), -1), (dict(o=P), -1), (dict(q=P + 8), -3),
    (dict(o=2 * P + 8), -3), (dict(lse=P + 1), -3), (dict(cu_seqlens=P + 1), -3)])
def test_paged_refusals(kw, code):
    assert _paged(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(cache=None), -1), (dict(cu_seqlens=0), -1), (dict(nseq=0), -1), (dict(total=0), -1),
    (dict(k_out=0, v_out=0), -1), (dict(k_out=2 * P, v_out=2 * P), -1), (dict(k_out=P), -1),
    (dict(v_out=P), -1), (dict(k_stride=255), -1), (dict(k_stride=128), -1), (dict(v_stride=0), -1),
    (dict(cache=_cache(d=96), k_stride=512, v_stride=512), -2), (dict(total=2 ** 30 + 1), -2),
    (dict(k_out=2 * P + 8), -3), (dict(v_out=3 * P + 2), -3), (dict(cu_seqlens=P + 2), -3)])
def test_read_refusals(kw, code):
    assert _read(**kw) == code


@pytest.mark.parametrize("max_q", [1, 3, 64])
def test_workspace(max_q):
    """Asked for with a bad shape it is 0; a call with less than it says is refused."""
    ask = gqa.gqa_attn_paged_q8_workspace_bytes
    assert ask(0, 1, 1, 1, 8, 2, 128) == 0 and ask(1, 1, 1, 1, 7, 2, 128) == 0
    assert ask(1, 1, 1, 1, 8, 2, 256) == 0 and ask(2, 64, max_q, 2 ** 30 + 1, 8, 2, 128) == 0
    n = ask(2, 2 * max_q, max_q, 60000, 8, 2, 128)
    assert n > 0 and n % 4 == 0
    kw = dict(total=2 * max_q, max_q=max_q, max_kv=60000,
              cache=_cache(max_pages=4000, num_pages=8000))
    assert _paged(workspace_bytes=n - 1, **kw) == -7
    assert _paged(workspace=0, **kw) == -7
    assert _paged(workspace=P + 8, workspace_bytes=n, **kw) == -3


def _tensors(**kw):
    t = dict(k=torch.zeros(4, 2, 16, 128, dtype=torch.uint8).view(torch.float8_e4m3fn),
             v=torch.zeros(4, 2, 16, 128, dtype=torch.uint8).view(torch.float8_e4m3fn),
             scales=torch.zeros(4, 2, 16, 2, dtype=torch.uint8).view(torch.float8_e8m0fnu),
             table=torch.zeros(3, 5, dtype=torch.int32), lens=torch.zeros(3, dtype=torch.int32))
    t.update(kw)
    return list(t.values())


def test_the_struct():
    ts = _tensors()
    a = gqa.make_paged_kv_q8(*ts)
    assert [int(a[n][0]) for n in ("num_pages", "Hkv", "page_size", "d", "max_pages")] == \
        [4, 2, 16, 128, 5]
    assert [int(a[n][0]) for n in ("k", "v", "scales", "page_table", "kv_lens")] == \
        [t.data_ptr() for t in ts]
    assert a.data_ptr() == a.ctypes.data


U8 = torch.zeros(4, 2, 16, 128, dtype=torch.uint8)


@pytest.mark.parametrize("kw", [
    dict(k=U8), dict(v=U8), dict(k=U8.view(torch.float8_e5m2)), dict(k=U8.bfloat16()),
    dict(k=U8[:3].view(torch.float8_e4m3fn)), dict(k=U8[0].view(torch.float8_e4m3fn)),
    dict(k=U8.view(torch.float8_e4m3fn).transpose(1, 2)),
    dict(scales=torch.zeros(4, 2, 16, 2, dtype=torch.uint8)),
    dict(scales=torch.zeros(4, 2, 16, 2)),
    dict(scales=torch.zeros(4, 2, 16, dtype=torch.uint8).view(torch.float8_e8m0fnu)),
    dict(scales=torch.zeros(4, 2, 16, 4, dtype=torch.uint8).view(torch.float8_e8m0fnu)[..., ::2]),
    dict(table=torch.zeros(3, 5, dtype=torch.int64)), dict(table=torch.zeros(5, dtype=torch.int32)),
    dict(lens=torch.zeros(2, dtype=torch.int32)), dict(lens=torch.zeros(3)),
    dict(lens=torch.zeros(3, dtype=torch.int32, device="meta")),
    dict(scales=torch.zeros(4, 2, 16, 2, dtype=torch.uint8, device="meta")
         .view(torch.float8_e8m0fnu))])
def test_tensors_that_do_not_fit(kw):
    with pytest.raises(ValueError):
        gqa.make_paged_kv_q8(*_tensors(**kw))


def _q8_layer():
    pool = torch.zeros(8, HKV, 16, D, dtype=torch.uint8).view(torch.float8_e4m3fn)
    return dataclasses.replace(
        _layer(), k_pool=pool, v_pool=pool.clone(),
        scales=torch.zeros(8, HKV, 16, 2, dtype=torch.uint8).view(torch.float8_e8m0fnu))


def test_a_stack_of_both_kinds():
    s = _stack([_layer(), _q8_layer()])
    assert s.caches[0].dtype == gqa.PAGED_KV_DTYPE and s.caches[1].dtype == gqa.PAGED_KV_Q8_DTYPE
    assert s.wsb >= gqa.gqa_attn_paged_q8_workspace_bytes(2, 6, 3, 32, 4, HKV, D)


def test_layers_that_do_not_fit():
    good = _q8_layer()
    for bad in (dataclasses.replace(good, scales=None),
                dataclasses.replace(_layer(), scales=good.scales),
                dataclasses.replace(good, scales=good.scales[:7]),
                dataclasses.replace(good, scales=torch.zeros(8, HKV, 16, 2, device="meta"))):
        with pytest.raises(ValueError):
            _stack([bad])
