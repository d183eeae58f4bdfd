"""The workspace query of the paged attention without a GPU: it answers for every shape, with 0
for the ones that the call refuses, and the call holds a workspace to its answer."""
import os
import subprocess
import sys

import numpy as np
import pytest

import global_causal_gqa_gb300 as gqa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000   # an aligned address that no call here dereferences
CODE = """
import global_causal_gqa_gb300 as gqa
for g in (65, 100, 127, 128, 129, 255, 256, 1 << 20, 2 ** 31 - 1):
    for max_q in (1, 2, 40):
        for nseq in (1, 2, 300):
            assert gqa.gqa_attn_paged_workspace_bytes(nseq, 300, max_q, 4096, g, 1, 128) == 0
for d in (1, 64, 127, 256, 512):
    for max_q in (1, 40):
        assert gqa.gqa_attn_paged_workspace_bytes(2, 80, max_q, 60000, 8, 2, d) == 0
assert gqa.gqa_attn_paged_workspace_bytes(2, 80, 41, 40, 8, 2, 128) == 0
print("answered")
"""


def _cache(Hkv):
    a = np.zeros(1, dtype=gqa.PAGED_KV_DTYPE)
    for n, x in dict(k=P, v=P, page_table=P, kv_lens=P, num_pages=8000, Hkv=Hkv, page_size=16,
                     d=128, max_pages=4000).items():
        a[n] = x
    return a


def test_refused_shapes_have_no_workspace():
    """In a process of its own: a group of more than 128 heads once divided by zero."""
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "answered", (r.returncode, r.stderr[-2000:])


@pytest.mark.parametrize("total,max_q", [(2, 1), (2, 2), (200, 100), (64, 40)])
def test_calls_hold_to_the_answer(total, max_q):
    """Split decode, drafts and split chunks: each needs a workspace, and less is refused."""
    n = gqa.gqa_attn_paged_workspace_bytes(2, total, max_q, 60000, 8, 2, 128)
    assert n > 0

    def call(workspace, size):
        return gqa.gqa_attn_paged(P, 1024, _cache(2), P, 2, total, max_q, 60000, 8, 0, 1.0, 2 * P,
                                  1024, P, workspace, size, stream=1, check=False)
    assert call(P, n - 1) == -7 and call(P, 0) == -7
    assert call(0, n) == -7 and call(P + 8, n) == -3
