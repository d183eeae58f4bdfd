"""Attention steps over every layer of a hybrid local/global decoder.

Decode over linear and ring caches (`LayerStack`):

"PLaMo 3アーキテクチャ徹底解析" §2.3 and §4.4: in a decode step each layer appends the new
token's K and V to its cache and attends over it; local layers keep a ring of the newest
W tokens, global layers a linear cache, in a fixed period (PLaMo 3: 7 local, then 1
global).  `LayerStack` drives that step through the C ABI: per layer one gqa_kv_append
and one gqa_attn_decode on a stream, with every layer's descriptor array in one device
buffer so that a whole step can be replayed from the same cache state (one copy restores
every layer's counts).  The step can be captured once in a CUDA graph and replayed.

Steps over paged caches (`PagedStack`): a packed batch of prompts, chunks, drafts and decode
tokens goes through each layer's QK norm + RoPE + append and its attention, local layers with
their window, over page tables that all layers share.

Argument marshalling and launch order only: every step of the computation runs in the
library's kernels.  The caller owns the caches, query and new-token tensors, outputs and
RoPE tables.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import List, Sequence

import numpy as np

from . import (KV_DESC_DTYPE, gqa_attn_decode, gqa_attn_paged, gqa_attn_paged_workspace_bytes,
               gqa_decode_workspace_bytes, gqa_kv_append, gqa_packed_rope_append, make_kv_descs,
               make_paged_kv)


@dataclass
class Layer:
    """One attention layer's caller-owned device tensors for a batch of nseq sequences."""
    k_cache: object        # [nseq, Hkv, cap, d] bf16
    v_cache: object        # [nseq, Hkv, cap, d] bf16
    q: object              # [nseq, Hq, d] bf16, the new query token
    k_new: object          # [nseq, Hkv, d] bf16, the new token's key (before RoPE)
    v_new: object          # [nseq, Hkv, d] bf16
    o: object              # [nseq, Hq, d] bf16, the attention output
    table: object          # RoPE table of the layer type, table_len positions
    table_len: int
    is_ring: bool          # local layer (ring of cap = W) or global (linear)
    count_before: Sequence[int]   # per sequence: tokens held (linear) / ever appended (ring)


class LayerStack:
    """Every layer's descriptors in one device buffer; `step` issues the decode step."""

    def __init__(self, layers: List[Layer], Hq: int, Hkv: int, d: int, scale: float,
                 max_len: int):
        import torch
        self.layers = layers
        self.Hq, self.Hkv, self.d, self.scale, self.max_len = Hq, Hkv, d, scale, max_len
        self.nseq = layers[0].q.shape[0]
        rows = []
        for L in layers:
            nseq, cap = L.k_cache.shape[0], L.k_cache.shape[2]
            a = make_kv_descs([L.k_cache[i] for i in range(nseq)],
                              [L.v_cache[i] for i in range(nseq)], [L.table] * nseq,
                              [cap] * nseq, list(L.count_before), [int(L.is_ring)] * nseq,
                              [L.table_len] * nseq)
            rows.append(torch.from_numpy(a.view(np.uint8).copy()))
        dev = layers[0].q.device
        self.descs0 = torch.stack(rows).to(dev)   # [layers, nseq * sizeof(gqa_kv_desc)]
        self.descs = self.descs0.clone()
        # a ring layer holds at most its capacity; a linear one at most max_len tokens
        self.max_lens = [L.k_cache.shape[2] if L.is_ring else max_len for L in layers]
        self.wsb = max(gqa_decode_workspace_bytes(self.nseq, Hq, Hkv, d, n)
                       for n in set(self.max_lens))
        self.ws = torch.empty(self.wsb, dtype=torch.uint8, device=dev)
        self.graph = None

    def restore(self):
        """Puts every layer's counts back to the state the stack was built with."""
        self.descs.copy_(self.descs0, non_blocking=True)

    def step(self, stream=None, restore: bool = True):
        """One decode step: (restore the counts,) then append + decode per layer."""
        if restore:
            self.restore()
        for l, L in enumerate(self.layers):
            gqa_kv_append(self.descs[l], self.nseq, L.k_new, L.v_new, self.Hkv, self.d, None,
                          stream)
            gqa_attn_decode(L.q, self.descs[l], self.nseq, self.Hq, self.Hkv, self.d,
                            self.scale, self.max_lens[l], L.o, None, self.ws, self.wsb, stream)

    def capture(self):
        """Captures `step` (with the count restore) in a CUDA graph on a side stream."""
        import torch
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                self.step()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = graph
        return graph

    def counts(self, layer: int) -> np.ndarray:
        a = self.descs[layer].cpu().numpy().view(KV_DESC_DTYPE)
        return a["count"].astype(np.int64)


@dataclass
class PagedLayer:
    """One attention layer's caller-owned device tensors for a packed batch of `total` tokens."""
    k_pool: object         # [num_pages, Hkv, page_size, d] bf16, keys after RoPE
    v_pool: object         # the same shape
    qkv: object            # [total, (Hq + 2 Hkv) d] bf16, rows of the fused projection
    o: object              # [total, Hq, d] bf16, the attention output
    q_gamma: object        # [d] float32 gains of the Q/K RMSNorm, or None
    k_gamma: object
    table: object          # RoPE table of the layer type, table_len positions
    table_len: int
    window: int            # 0: global layer


class PagedStack:
    """A serving step over paged caches: per layer one gqa_packed_rope_append and one
    gqa_attn_paged.  cu_seqlens (int32 [nseq + 1]), kv_lens (int32 [nseq], counted with the new
    tokens) and page_table (int32 [nseq, max_pages], used by every layer with its own pools)
    are device tensors read when the kernels run: a captured step follows what the caller
    writes to them between replays, up to max_q new tokens and max_kv tokens of a sequence.
    Chunks run fastest with a max_kv near the longest sequence.  A stack has one workspace and
    one tensor of rotated queries: its steps, eager or replayed, must not overlap."""

    def __init__(self, layers: List[PagedLayer], cu_seqlens, kv_lens, page_table, max_q: int,
                 max_kv: int, Hq: int, Hkv: int, d: int, scale: float, eps: float = 1e-6):
        import torch
        self.layers, self.cu_seqlens, self.kv_lens = layers, cu_seqlens, kv_lens
        self.page_table = page_table
        self.max_q, self.max_kv, self.Hq, self.Hkv, self.d = max_q, max_kv, Hq, Hkv, d
        self.scale, self.eps = scale, eps
        self.nseq, self.total = page_table.shape[0], layers[0].qkv.shape[0]
        if cu_seqlens.shape != (self.nseq + 1,) or cu_seqlens.dtype != torch.int32 or \
                not cu_seqlens.is_contiguous():
            raise ValueError("PagedStack: cu_seqlens is contiguous int32 [nseq + 1]")
        for i, L in enumerate(layers):
            if any(t is not None and t.device != page_table.device for t in
                   (cu_seqlens, L.k_pool, L.qkv, L.o, L.q_gamma, L.k_gamma, L.table)):
                raise ValueError(f"PagedStack: layer {i}: the tensors lie on one device")
            for t, name, shape in ((L.qkv, "qkv", (self.total, (Hq + 2 * Hkv) * d)),
                                   (L.o, "o", (self.total, Hq, d))):
                if tuple(t.shape) != shape or t.dtype != torch.bfloat16 or not t.is_contiguous():
                    raise ValueError(f"PagedStack: layer {i}: {name} is contiguous bfloat16 "
                                     f"{list(shape)}")
            if L.k_pool.shape[1] != Hkv or L.k_pool.shape[3] != d:
                raise ValueError(f"PagedStack: layer {i}: pools of {Hkv} KV heads of {d}")
            for t, name, n in ((L.q_gamma, "q_gamma", d), (L.k_gamma, "k_gamma", d),
                               (L.table, "table", L.table_len * d)):
                if t is not None and (t.numel() < n or t.dtype != torch.float32 or
                                      not t.is_contiguous()):
                    raise ValueError(f"PagedStack: layer {i}: {name} is contiguous float32, "
                                     f"{n} values")
        self.caches = [make_paged_kv(L.k_pool, L.v_pool, page_table, kv_lens) for L in layers]
        dev = layers[0].qkv.device
        self.wsb = gqa_attn_paged_workspace_bytes(self.nseq, self.total, max_q, max_kv, Hq, Hkv, d)
        self.ws = torch.empty(max(self.wsb, 16), dtype=torch.uint8, device=dev)
        self.q = torch.empty(self.total, Hq, d, dtype=torch.bfloat16, device=dev)
        self.graph = None

    def step(self, stream=None):
        """One step: every layer appends its new tokens' keys and values, then attends."""
        Hq, Hkv, d = self.Hq, self.Hkv, self.d
        row = (Hq + 2 * Hkv) * d
        for L, cache in zip(self.layers, self.caches):
            q, k, v = L.qkv.split([Hq * d, Hkv * d, Hkv * d], 1)
            gqa_packed_rope_append(q, row, k, row, v, row, self.cu_seqlens, self.nseq, self.total,
                                   Hq, Hkv, d, L.q_gamma, L.k_gamma, self.eps, L.table,
                                   L.table_len, self.q, None, cache, stream)
            gqa_attn_paged(self.q, Hq * d, cache, self.cu_seqlens, self.nseq, self.total,
                           self.max_q, self.max_kv, Hq, L.window, self.scale, L.o, Hq * d, None,
                           self.ws, self.wsb, stream)

    def capture(self):
        """Captures `step` in a CUDA graph on a side stream (run `step` once before: the first
        call of a kernel loads it)."""
        import torch
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                self.step()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = graph
        return graph
