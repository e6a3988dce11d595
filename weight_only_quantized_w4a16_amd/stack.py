"""Token-by-token decode through a stack of LLaMA-style quantised linear layers.

The pages measure generation speed in iterations per second of a whole model
(Triton GPTQ page, "Highlighted Details": LLaMA-7B, 4-bit against GPTQ CUDA
and FP16) and observe that decode is matrix-vector work bound by memory
bandwidth (exllama bandwidth discussion, GPTQ quote and turboderp's reply).
This module chains the library's entry points the way one decoder layer uses
its linear layers -- fused QKV, output projection, activation-fused gate+up,
down projection -- over many layers, so a step is one token through every
layer's weights.

DecodeStack is the chain of products alone: attention, normalisation and the
residual path are not weight-only-quantised products and are not modelled, the
first `dim` columns of the QKV output stand in for the attention output that
feeds the output projection.  CachedStack adds what surrounds the products: keys
and values quantised into a 4-bit paged cache per layer, attention over it, the
QKV bias and the residual path in the products' epilogues, and where they are
given the norms before the products, rotary positions on queries and keys, and
low-rank adapters beside the QKV, output and down projections.

Only argument marshalling and sequencing live here; every product runs in the
library's kernels.  All buffers are allocated once, so a step launches exactly
four kernels per layer (plus one copy per layer when M > 1, where the QKV
slice is not contiguous) and can be captured in a HIP graph.
"""
from __future__ import annotations

import dataclasses
from typing import List, Optional, Tuple

import torch

from . import (KVCache, KVPages, LoraBank, PackedLayer, Rotary, linear, use_gemv, wq_gemm, wq_gemm_gate_up, wq_gemv,
               wq_gemv_gate_up, _empty, wq_kv_attention, wq_kv_cache, wq_kv_pages, wq_kv_workspace_bytes, wq_kv_write, wq_lora,
               wq_lora_workspace_bytes, wq_rms_norm, wq_rotary)


@dataclasses.dataclass
class DecoderWeights:
    """The four repacked linear layers of one decoder layer."""
    qkv: PackedLayer       # [dim] -> [3 * dim] (fused Q, K, V)
    o: PackedLayer         # [dim] -> [dim]
    gate_up: PackedLayer   # [dim] -> [2 * inter], repacked by wq_repack_gate_up
    down: PackedLayer      # [inter] -> [dim]


def _copies(stream, **tensors) -> dict:
    """Clones made on `stream` (the current one by default), where the work that fills the tensors is."""
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        copies = {name: t.clone() for name, t in tensors.items()}
    for t in copies.values():
        t.record_stream(here)
    return copies


class DecodeStack:
    """y = layer_L-1( ... layer_0(x)) with layer(x) = down(SiLU(gate(o(qkv(x)[:, :dim]))) * up(...))."""

    def __init__(self, layers: List[DecoderWeights], M: int, dtype: torch.dtype, device):
        if not layers:
            raise ValueError("empty stack")
        l0 = layers[0]
        self.dim, self.inter = l0.o.K, l0.down.K
        for L in layers:
            if not L.gate_up.gate_up:
                raise ValueError("gate_up must be repacked by wq_repack_gate_up")
            if (L.qkv.K, L.o.K, L.o.N, L.gate_up.K, L.gate_up.N, L.down.K, L.down.N) != \
                    (self.dim, self.dim, self.dim, self.dim, 2 * self.inter, self.inter, self.dim):
                raise ValueError("layer shapes do not chain")
            if L.qkv.N < self.dim:
                raise ValueError("the QKV output must hold at least dim columns")
        self.layers = layers
        self.M = M
        small = all(use_gemv(M, lay) for L in layers for lay in (L.qkv, L.o, L.gate_up, L.down))
        self._lin = wq_gemv if small else wq_gemm
        self._lin_gu = wq_gemv_gate_up if small else wq_gemm_gate_up
        e = dict(dtype=dtype, device=device)
        self.qkv_out = torch.empty((M, l0.qkv.N), **e)
        self.attn = torch.empty((M, self.dim), **e)
        self.o_out = torch.empty((M, self.dim), **e)
        self.h = torch.empty((M, self.inter), **e)
        self.x = [torch.empty((M, self.dim), **e), torch.empty((M, self.dim), **e)]

    def step(self, x: torch.Tensor, stream=None, record: Optional[list] = None) -> torch.Tensor:
        """One token (M rows) through every layer on `stream` (a torch stream; the
        current one by default); returns the last layer's output (a buffer of the
        stack, overwritten by the next step).  With `record`, the input and output
        of every product are appended as tensors (clones)."""
        if x.shape != (self.M, self.dim) or not x.is_contiguous():
            raise ValueError("x must be a contiguous [M][dim] tensor")
        cur = x
        for i, L in enumerate(self.layers):
            if record is not None:  # (the layer's output may be written over its input)
                record.append(dict(layer=i, **_copies(stream, x=cur)))
            self._lin(cur, L.qkv, out=self.qkv_out, stream=stream)
            if self.M == 1:
                attn = self.qkv_out[:, :self.dim]  # a contiguous prefix of the single row
            else:
                attn = self.attn
                with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
                    attn.copy_(self.qkv_out[:, :self.dim])
            self._lin(attn, L.o, out=self.o_out, stream=stream)
            self._lin_gu(self.o_out, L.gate_up, out=self.h, stream=stream)
            nxt = self.x[i % 2]
            self._lin(self.h, L.down, out=nxt, stream=stream)
            if record is not None:
                record[-1].update(_copies(stream, qkv=self.qkv_out, attn=attn, o=self.o_out, h=self.h, y=nxt))
            cur = nxt
        return cur


@dataclasses.dataclass
class LayerAdapters:
    """The adapters of one decoder layer's products (None: that product has none).  The gate+up product applies its
    activation in its epilogue, which takes no adapter: variants that adapt those two projections do not run here."""
    qkv: Optional[LoraBank] = None    # three slices: queries, keys, values (or one)
    o: Optional[LoraBank] = None
    down: Optional[LoraBank] = None


class CachedStack:
    """Layers of attention over a 4-bit cache and a gated feed-forward product, each on a residual path:
    x1 = x + o(attention(rotary(qkv(norm(x)) + bias))), y = x1 + down(SiLU(gate(norm(x1))) * up(norm(x1))).

    norms: two weights [dim] per layer, before QKV and before gate+up (None: no norms); eps theirs.  rotary: turns
    queries and keys to their rows' positions (None: not at all).  adapters: low-rank adapters per layer, of which each
    sequence of a step names its own; their part is added to the product as it was stored (bias and residual with it),
    so these rows are rounded twice.

    A step takes the rows of any number of sequences -- prompts, chunks of them or single tokens -- named as
    everywhere in the cache's functions: block_table, kv_lens (with the step's rows) and cu_q (None: as many rows
    each).  The page tables are the caller's; all layers use the same ones, each on a cache of its own."""

    def __init__(self, layers: List[DecoderWeights], q_heads: int, kv_heads: int, head_dim: int, num_pages: int,
                 max_rows: int, dtype: torch.dtype, device, page_size: int = 16, group: Optional[int] = None,
                 qkv_bias: Optional[List[torch.Tensor]] = None,
                 norms: Optional[List[Tuple[torch.Tensor, torch.Tensor]]] = None, eps: float = 1e-6,
                 rotary: Optional[Rotary] = None, adapters: Optional[List[LayerAdapters]] = None):
        if not layers:
            raise ValueError("empty stack")
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.dim, self.inter = layers[0].qkv.K, layers[0].down.K
        qkv_n, attn_n = (q_heads + 2 * kv_heads) * head_dim, q_heads * head_dim
        for L in layers:
            if not L.gate_up.gate_up:
                raise ValueError("gate_up must be repacked by wq_repack_gate_up")
            if (L.qkv.K, L.qkv.N, L.o.K, L.o.N, L.gate_up.K, L.gate_up.N, L.down.K, L.down.N) != \
                    (self.dim, qkv_n, attn_n, self.dim, self.dim, 2 * self.inter, self.inter, self.dim):
                raise ValueError("layer shapes do not chain")
        if qkv_bias is not None and len(qkv_bias) != len(layers):
            raise ValueError("one QKV bias per layer")
        if norms is not None and len(norms) != len(layers):
            raise ValueError("two norm weights per layer")
        if rotary is not None and rotary.head_dim != head_dim:
            raise ValueError("the rotary plan is one of other heads")
        if adapters is not None:
            if len(adapters) != len(layers):
                raise ValueError("one set of adapters per layer")
            for L, A in zip(layers, adapters):
                for bank, lay in ((A.qkv, L.qkv), (A.o, L.o), (A.down, L.down)):
                    if bank is not None and (bank.K, bank.N) != (lay.K, lay.N):
                        raise ValueError("adapters of other products")
        if max_rows < 1:
            raise ValueError("max_rows must be positive")
        self.norms, self.eps, self.rotary, self.adapters = norms, eps, rotary, adapters
        self.layers, self.bias, self.max_rows = layers, qkv_bias, max_rows
        group = group or min(128, head_dim & -head_dim)
        self.caches: List[KVCache] = [wq_kv_cache(num_pages, page_size, kv_heads, head_dim, group, dtype, device)
                                      for _ in layers]
        e = dict(dtype=dtype, device=device)
        self.qkv_out = torch.empty((max_rows, qkv_n), **e)
        self.attn = torch.empty((max_rows, q_heads, head_dim), **e)
        self.mid = torch.empty((max_rows, self.dim), **e)
        self.h = torch.empty((max_rows, self.inter), **e)
        self.x = [torch.empty((max_rows, self.dim), **e), torch.empty((max_rows, self.dim), **e)]
        self.normed = torch.empty((max_rows, self.dim), **e) if norms is not None else None

    def pages(self, batch: int, max_pages: int) -> KVPages:
        """Page tables of `batch` empty sequences over the stack's caches, for wq_kv_resize."""
        c = self.caches[0]
        return wq_kv_pages(c.num_pages, c.page_size, batch, max_pages, c.data.device)

    def step(self, x: torch.Tensor, block_table: torch.Tensor, kv_lens: torch.Tensor,
             cu_q: Optional[torch.Tensor] = None, max_kv_len: Optional[int] = None, window: int = 0, stream=None,
             record: Optional[list] = None, adapters: Optional[torch.Tensor] = None,
             positions: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The rows x [rows][dim] through every layer; returns the last layer's output (a buffer of the stack,
        overwritten by the next step).  max_kv_len as for wq_kv_attention.  adapters: int32 [batch], each sequence's
        adapter (a stack with adapters needs it).  positions: as for wq_rotary (default: those of the sequences).  With
        `record`, the inputs and outputs of every part are appended as tensors (clones)."""
        T = x.shape[0]
        if x.dim() != 2 or x.shape[1] != self.dim or not x.is_contiguous() or T > self.max_rows:
            raise ValueError("x must be a contiguous [rows][dim] tensor of at most max_rows rows")
        H, KV, D = self.q_heads, self.kv_heads, self.head_dim
        qkv, attn, mid, h = self.qkv_out[:T], self.attn[:T], self.mid[:T], self.h[:T]
        heads = qkv.view(T, H + 2 * KV, D)
        q, k, v = heads[:, :H], heads[:, H:H + KV], heads[:, H + KV:]
        batch, ragged = block_table.shape[0], cu_q is not None
        need = wq_kv_workspace_bytes(T, batch, ragged, H, KV, D, self.caches[0].group,
                                     block_table.shape[1] * self.caches[0].page_size if max_kv_len is None
                                     else max_kv_len)
        ws = _empty(stream, x, need, torch.uint8, scratch=True) if need else None
        if (self.adapters is None) != (adapters is None):
            raise ValueError("a stack with adapters, and no other, needs each sequence's adapter")
        if adapters is not None and adapters.shape != kv_lens.shape:
            raise ValueError(f"{kv_lens.shape[0]} sequences need as many adapters, got {tuple(adapters.shape)}")
        if positions is not None and self.rotary is None:
            raise ValueError("positions are for a stack with rotary positions")
        lora_ws = None
        if adapters is not None:
            banks = [b for A in self.adapters for b in (A.qkv, A.o, A.down) if b is not None]
            most = max((wq_lora_workspace_bytes(T, batch, b.K, b.rank, b.num_slices) for b in banks), default=0)
            lora_ws = _empty(stream, x, most, torch.uint8, scratch=True) if most else None

        def adapt(bank, inp, out):
            if bank is not None:
                wq_lora(inp, bank, adapters, out, cu_q, out=out, ws=lora_ws, stream=stream)

        none = LayerAdapters()
        cur = x
        for i, (L, cache) in enumerate(zip(self.layers, self.caches)):
            A = none if adapters is None else self.adapters[i]
            if record is not None:  # (the layer's output may be written over its input)
                record.append(dict(layer=i, **_copies(stream, x=cur)))
            inp = cur
            if self.norms is not None:
                inp = wq_rms_norm(cur, self.norms[i][0], self.eps, out=self.normed[:T], stream=stream)
                if record is not None:
                    record[-1].update(_copies(stream, n1=inp))
            linear(inp, L.qkv, out=qkv, stream=stream, bias=None if self.bias is None else self.bias[i])
            adapt(A.qkv, inp, qkv)
            if self.rotary is not None:
                if record is not None:
                    record[-1].update(_copies(stream, unturned=qkv))
                if positions is not None:
                    wq_rotary(q, k, self.rotary, positions, out=(q, k), stream=stream)
                else:
                    wq_rotary(q, k, self.rotary, kv_lens=kv_lens, cu_q=cu_q, out=(q, k), stream=stream)
            wq_kv_write(k, v, cache, block_table, kv_lens, cu_q, stream=stream)
            wq_kv_attention(q, cache, block_table, kv_lens, cu_q, window=window, max_kv_len=max_kv_len, out=attn,
                            ws=ws, stream=stream)
            linear(attn.view(T, H * D), L.o, out=mid, stream=stream, residual=cur)
            adapt(A.o, attn.view(T, H * D), mid)
            inp = mid
            if self.norms is not None:
                inp = wq_rms_norm(mid, self.norms[i][1], self.eps, out=self.normed[:T], stream=stream)
                if record is not None:
                    record[-1].update(_copies(stream, n2=inp))
            linear(inp, L.gate_up, out=h, stream=stream)
            nxt = self.x[i % 2][:T]
            linear(h, L.down, out=nxt, stream=stream, residual=mid)
            adapt(A.down, h, nxt)
            if record is not None:
                record[-1].update(_copies(stream, qkv=qkv, attn=attn, mid=mid, h=h, y=nxt))
            cur = nxt
        return cur
