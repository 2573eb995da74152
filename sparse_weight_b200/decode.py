"""The attention block of a decode (or prefill) step over an 8-bit cache.

    q, k, v = Wq x, Wk x, Wv x          the library's products
    cache  <- k, v                       hyb_cache_append
    a       = attention(q, cache)        hyb_cache_attention
    y       = Wo a                       the library's products

Each weight is a tile-hybrid matrix (``hyb.Packed``) or an 8-bit one
(``hyb.Fp8Matrix``); mixing them in one block is fine.  The block owns the
workspaces of its calls, sized once for the largest step, so a step allocates
only its activations and can be captured in a CUDA graph.  Steps of one block
run one after another on one stream (they share the workspaces and write the
cache).
"""
from typing import Callable, Optional, Union

import torch

from . import hyb

Weight = Union[hyb.Packed, hyb.Fp8Matrix]


class AttentionBlock:
    """heads query heads over kv_heads cached ones; the cache gives head_dim.

    max_rows, max_new, max_batch and max_pages bound the steps: new tokens in
    all, new tokens of one sequence, sequences, and pages per sequence."""

    def __init__(self, wq: Weight, wk: Weight, wv: Weight, wo: Weight, heads: int,
                 cache: hyb.Cache, max_batch: int, max_pages: int, max_new: int = 1,
                 max_rows: Optional[int] = None, window: int = 0, sinks: int = 0):
        self.wq, self.wk, self.wv, self.wo = wq, wk, wv, wo
        self.heads, self.cache, self.window, self.sinks = heads, cache, window, sinks
        self.max_batch, self.max_pages, self.max_new = max_batch, max_pages, max_new
        self.max_rows = max_batch * max_new if max_rows is None else max_rows
        kv_heads, dim = cache.k.shape[1], cache.k.shape[3]
        for name, w, rows in (("wq", wq, heads * dim), ("wk", wk, kv_heads * dim),
                              ("wv", wv, kv_heads * dim)):
            if w.n != rows or w.k != wq.k:
                raise ValueError(f"AttentionBlock: {name} must be [{rows}][{wq.k}], "
                                 f"got [{w.n}][{w.k}]")
        if wo.k != heads * dim:
            raise ValueError(f"AttentionBlock: wo must have {heads * dim} inputs, got {wo.k}")
        dev = cache.k.device
        weights = (wq, wk, wv, wo)
        packed = [w for w in weights if isinstance(w, hyb.Packed)]
        eight = [w for w in weights if isinstance(w, hyb.Fp8Matrix)]
        self._ws_skinny = self._ws_prefill = self._ws_fp8 = self._ws_quant = None
        if packed:
            self._ws_skinny = hyb.new_workspace(
                max(hyb.workspace_bytes(w, b) for w in packed
                    for b in range(1, min(16, self.max_rows) + 1)), dev)
            if self.max_rows > 16:
                self._ws_prefill = hyb.new_workspace(
                    int(hyb.lib().hyb_prefill_workspace_bytes()), dev)
        if eight:
            self._ws_fp8 = hyb.new_workspace(
                max(hyb.fp8_workspace_bytes(m, w.n, w.k) for w in eight
                    for m in {min(16, self.max_rows), self.max_rows}), dev)
            self._ws_quant = hyb.new_workspace(hyb.fp8_quant_workspace_bytes(), dev)
        self._ws_append = hyb.new_workspace(hyb.cache_append_workspace_bytes(), dev)
        self._ws_attention = hyb.new_workspace(
            hyb.cache_attention_workspace_bytes(cache, max_batch, heads, max_new,
                                                max_pages * cache.page_size), dev)

    def _product(self, w: Weight, x: torch.Tensor, xs=None, xq=None) -> torch.Tensor:
        if isinstance(w, hyb.Fp8Matrix):
            if xq is not None:
                return hyb.matmul_fp8(w, xq, xs=xs, ydt=hyb.HYB_BF16, ws=self._ws_fp8)
            return hyb.matmul_fp8(w, x, ydt=hyb.HYB_BF16, ws=self._ws_fp8)
        if x.shape[0] <= 16:
            return hyb.spmm_skinny(w, x, ydt=hyb.HYB_BF16, ws=self._ws_skinny)
        return hyb.spmm_prefill(w, x, ws=self._ws_prefill).to(torch.bfloat16)

    def step(self, x: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
             off: Optional[torch.Tensor] = None, max_new: Optional[int] = None,
             rotate: Optional[Callable] = None) -> torch.Tensor:
        """One step: x bf16 [rows][k] holds the new tokens of all sequences,
        lens their lengths with them (see hyb.cache_append); max_new is the most
        of one sequence (by default rows / batch, with off the block's).  ``rotate(q, k)``
        may return position-dependent q [rows][heads][dim] and k
        [rows][kv_heads][dim].  Returns bf16 [rows][wo.n].

        With off, rows behind the last sequence (off[batch] .. rows - 1: a step of
        a fixed size that is not full) get the output of a zero attention.  x is
        multiplied there too: keep it finite, as elsewhere."""
        rows = x.shape[0]
        batch, pages = page_table.shape
        if max_new is not None:
            new = max_new
        else:  # with off, any sequence may have as many as the block allows
            new = rows // max(batch, 1) if off is None else self.max_new
        if rows > self.max_rows or batch > self.max_batch or pages > self.max_pages \
                or new > self.max_new:
            raise ValueError("AttentionBlock: the step is larger than the block was made for")
        kv_heads, dim = self.cache.k.shape[1], self.cache.k.shape[3]
        # the attention leaves rows of no sequence as they were, and the last product reads them
        a = None if off is None else torch.zeros(rows, self.heads, dim, dtype=torch.bfloat16, device=x.device)
        xq = xs = None
        if rows > 16 and sum(isinstance(w, hyb.Fp8Matrix) for w in (self.wq, self.wk, self.wv)) > 1:
            xq, xs = hyb.quant_fp8(x, ws=self._ws_quant)  # once for the products that share x
        q = self._product(self.wq, x, xs, xq).view(rows, self.heads, dim)
        k = self._product(self.wk, x, xs, xq).view(rows, kv_heads, dim)
        v = self._product(self.wv, x, xs, xq).view(rows, kv_heads, dim)
        if rotate is not None:
            q, k = rotate(q, k)
        hyb.cache_append(self.cache, k, v, page_table, lens, off, new, ws=self._ws_append)
        a = hyb.cache_attention(self.cache, q, page_table, lens, off, new, window=self.window,
                                sinks=self.sinks, out=a, ws=self._ws_attention)
        return self._product(self.wo, a.view(rows, self.heads * dim))

    def check(self) -> None:
        """Synchronise and raise if a kernel of the steps so far flagged a problem."""
        for ws in (self._ws_skinny, self._ws_prefill, self._ws_fp8, self._ws_quant,
                   self._ws_append, self._ws_attention):
            if ws is not None:
                hyb.check_status(ws)
