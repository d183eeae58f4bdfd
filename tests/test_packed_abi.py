"""The packed and paged entry points without a GPU: wrong arguments are refused on the host
before anything is launched, and the workspace sizes follow from the shape."""
import numpy as np
import pytest

import global_causal_gqa_gb300 as gqa

P = 0x10000   # an aligned address that no call here dereferences


def _cache(**kw):
    a = np.zeros(1, dtype=gqa.PAGED_KV_DTYPE)
    f = dict(k=P, v=P, page_table=P, kv_lens=P, num_pages=4, Hkv=2, page_size=16, d=128,
             max_pages=2, reserved=0)
    f.update(kw)
    for n, x in f.items():
        a[n] = x
    return a


def _packed(**kw):
    a = dict(q=P, q_stride=1024, k=P, k_stride=256, v=P, v_stride=256, o=2 * P, o_stride=1024,
             lse=P, cu_seqlens=P, nseq=2, total=10, Hq=8, Hkv=2, d=128, window=0, scale=1.0)
    a.update(kw)
    return gqa.gqa_attn_packed(*a.values(), stream=1, check=False)


def _append(**kw):
    a = dict(q=P, q_stride=1024, k=P, k_stride=256, v=P, v_stride=256, cu_seqlens=P, nseq=2,
             total=10, Hq=8, Hkv=2, d=128, q_gamma=P, k_gamma=P, eps=1e-6, table=P, table_len=64,
             q_out=2 * P, k_out=3 * P, cache=_cache())
    a.update(kw)
    return gqa.gqa_packed_rope_append(*a.values(), stream=1, check=False)


def _paged(**kw):
    a = dict(q=P, q_stride=1024, cache=_cache(), cu_seqlens=P, nseq=2, total=10, max_q=5,
             max_kv=32, Hq=8, window=0, scale=1.0, o=2 * P, o_stride=1024, lse=P, workspace=P,
             workspace_bytes=1 << 40)
    a.update(kw)
    return gqa.gqa_attn_paged(*a.values(), stream=1, check=False)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(o=0), -1), (dict(cu_seqlens=0), -1),
    (dict(nseq=0), -1), (dict(total=0), -1), (dict(total=-5), -1), (dict(Hq=0), -1),
    (dict(Hkv=0), -1), (dict(Hkv=3), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=NAN), -1), (dict(scale=INF), -1), (dict(d=64), -2), (dict(d=256), -2),
    (dict(Hq=130, Hkv=2, q_stride=130 * 128, o_stride=130 * 128), -2),
    (dict(q_stride=1016), -1), (dict(k_stride=248), -1), (dict(v_stride=128), -1),
    (dict(o_stride=1028), -1), (dict(q_stride=-1024), -1), (dict(o=P), -1),
    (dict(q=P + 8), -3), (dict(v=P + 2), -3), (dict(lse=P + 2), -3), (dict(cu_seqlens=P + 1), -3),
])
def test_packed_refusals(kw, code):
    assert _packed(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), -1), (dict(q=0), -1), (dict(q_out=0), -1), (dict(v=0), -1), (dict(table=0), -1),
    (dict(cu_seqlens=0), -1), (dict(q=0, q_out=0, k_out=0, cache=None), -1),
    (dict(nseq=0), -1), (dict(total=0), -1), (dict(Hq=0), -1), (dict(Hkv=0), -1),
    (dict(table_len=0), -1), (dict(eps=-1.0), -1), (dict(eps=NAN), -1), (dict(eps=INF), -1),
    (dict(d=96), -2), (dict(q_stride=1020), -1), (dict(k_stride=128), -1), (dict(v_stride=0), -1),
    (dict(q_out=P, q_stride=1032), -1), (dict(k_out=P, k_stride=264), -1),
    (dict(q=P + 4), -3), (dict(k_out=P + 4), -3), (dict(q_gamma=P + 4), -3), (dict(table=P + 8), -3),
    (dict(cu_seqlens=P + 2), -3), (dict(cache=_cache(k=0)), -1), (dict(cache=_cache(kv_lens=0)), -1),
    (dict(cache=_cache(num_pages=0)), -1), (dict(cache=_cache(max_pages=0)), -1),
    (dict(cache=_cache(reserved=1)), -1), (dict(cache=_cache(page_size=24)), -2),
    (dict(cache=_cache(page_size=256)), -2), (dict(cache=_cache(Hkv=1)), -1),
    (dict(cache=_cache(d=64)), -1), (dict(cache=_cache(v=P + 8)), -3),
    (dict(cache=_cache(page_table=P + 2)), -3),
])
def test_append_refusals(kw, code):
    assert _append(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), -1), (dict(cache=None), -1), (dict(o=0), -1), (dict(cu_seqlens=0), -1),
    (dict(nseq=0), -1), (dict(total=0), -1), (dict(max_q=0), -1), (dict(max_kv=4), -1),
    (dict(Hq=0), -1), (dict(Hq=7), -1), (dict(scale=0.0), -1), (dict(scale=NAN), -1),
    (dict(cache=_cache(d=256), q_stride=2048, o_stride=2048), -2), (dict(cache=_cache(page_size=8)), -2),
    (dict(Hq=130, q_stride=130 * 128, o_stride=130 * 128), -2),
    (dict(q_stride=1022), -1), (dict(o_stride=512), -1), (dict(o=P), -1), (dict(q=P + 8), -3),
    (dict(lse=P + 1), -3), (dict(cache=_cache(k=P + 8)), -3), (dict(cache=_cache(kv_lens=P + 1)), -3),
    (dict(cache=_cache(Hkv=0)), -1),
])
def test_paged_refusals(kw, code):
    assert _paged(**kw) == code


def test_paged_workspace():
    """Asked for with a bad shape it is 0; a call with less than it says is refused."""
    assert gqa.gqa_attn_paged_workspace_bytes(0, 1, 1, 1, 8, 2, 128) == 0
    assert gqa.gqa_attn_paged_workspace_bytes(1, 1, 1, 1, 7, 2, 128) == 0
    n = gqa.gqa_attn_paged_workspace_bytes(2, 2, 1, 60000, 8, 2, 128)
    if n:
        cache = _cache(max_pages=4000, num_pages=8000)
        kw = dict(total=2, max_q=1, max_kv=60000, cache=cache)
        assert _paged(workspace_bytes=n - 1, **kw) == -7
        assert _paged(workspace=0, **kw) == -7
        assert _paged(workspace=P + 8, workspace_bytes=n, **kw) == -3


def test_make_paged_kv_checks_its_tensors():
    import torch
    k = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    t, n = torch.zeros(3, 5, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    a = gqa.make_paged_kv(k, k.clone(), t, n)
    assert (int(a["num_pages"][0]), int(a["Hkv"][0]), int(a["page_size"][0]), int(a["d"][0]),
            int(a["max_pages"][0])) == (4, 2, 16, 128, 5)
    assert int(a["k"][0]) == k.data_ptr() and int(a["kv_lens"][0]) == n.data_ptr()
    for bad in ((k.transpose(1, 2), k, t, n), (k, k[:3], t, n), (k.float(), k.float(), t, n),
                (k, k, t.long(), n), (k, k, t, n[:2]), (k, k, t[0], n)):
        with pytest.raises(ValueError):
            gqa.make_paged_kv(*bad)
