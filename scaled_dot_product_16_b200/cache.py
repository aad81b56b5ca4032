"""A paged key/value cache for serving: the page table, its pages and the calls that work on them.

`PagedCache` holds what a program that answers with a model keeps between its steps: a pool of pages of
keys and values for each layer, one page table, reference counts and lengths for all layers, and the
buffers that the calls need. It only owns device memory and marshals it into the library's calls; what
happens to it is decided on the device (no method waits for the GPU, except check()), so that a step of
reserve, append and attend can be captured into a CUDA graph and replayed.

    cache = PagedCache(layers=32, rows=64, max_pages=512, num_pages=20000, page_size=16, Nq=32, Nkv=8, D=128,
                       dtype=ATTN_BF16, device="cuda")
    cache.reserve(new_tokens)                                    # pages for the prompts' tokens
    for layer in range(32):
        cache.prefill(layer, q, k, v, cu_seqlens, out)           # attention of the prompts, into the cache
    while ...:
        cache.reserve(live_only=True)                            # one more token per row that has not ended
        for layer in range(32):
            cache.append(layer, k, v)
            cache.attend(layer, q, out)
        cache.fork(parents)                                      # beam search; or -1 for rows that are done
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (ATTN_BF16, ATTN_BHSD, ATTN_F16, ATTN_F32, ATTN_OK, ATTN_TND, ATTN_WINDOW_ALL, AttnError,
               attn_cache_append, attn_cache_compact, attn_cache_copy, attn_cache_evict, attn_cache_fork,
               attn_cache_grow, attn_decode_paged, attn_decode_workspace_size, attn_fwd_sinks,
               attn_get_last_error)

_DTYPE = {ATTN_BF16: torch.bfloat16, ATTN_F32: torch.float32, ATTN_F16: torch.float16}


class PagedCache:
    """See the module's description. Every query sees the keys that attn_fwd_sinks's rule gives it with
    `window_tokens` and `sink_tokens`. Rows are empty at first; a row of length 0 takes part in every call
    and costs next to nothing. Calls that overlap on the device (other streams) need caches of their
    own."""

    def __init__(self, *, layers: int, rows: int, max_pages: int, num_pages: int, page_size: int, Nq: int, Nkv: int,
                 D: int, dtype: int = ATTN_BF16, layout: int = ATTN_TND, scale: Optional[float] = None,
                 window_tokens: int = ATTN_WINDOW_ALL, sink_tokens: int = 0, device="cuda"):
        self.layers, self.rows, self.max_pages, self.num_pages, self.page_size = layers, rows, max_pages, num_pages, page_size
        self.Nq, self.Nkv, self.D, self.dtype, self.layout = Nq, Nkv, D, dtype, layout
        self.scale = D ** -0.5 if scale is None else scale
        self.window_tokens, self.sink_tokens = window_tokens, sink_tokens
        page = (Nkv, page_size, D) if layout == ATTN_BHSD else (page_size, Nkv, D)
        self.pool = torch.empty((layers, 2, num_pages, *page), dtype=_DTYPE[dtype], device=device)
        i32 = dict(dtype=torch.int32, device=device)
        self.page_table = torch.full((rows, max_pages), -1, **i32)
        self.ref_count = torch.zeros(num_pages, **i32)
        self.seq_lens = torch.zeros(rows, **i32)
        self.new_lens = torch.zeros(rows, **i32)  # lengths of the rows that the last reserve gave tokens, else 0
        self._copies = torch.empty((rows, 2), **i32)
        self._moves = torch.empty((max(1, num_pages // 2), 2), **i32)
        self.page_map = torch.empty(num_pages, **i32)
        self.live_pages = torch.zeros(1, **i32)
        self.workspace = torch.zeros(attn_decode_workspace_size(Nq=Nq, Nkv=Nkv, D=D, dtype=dtype), dtype=torch.uint8,
                                     device=device)

    def _sizes(self):
        return dict(Nkv=self.Nkv, D=self.D, num_pages=self.num_pages, page_size=self.page_size, max_pages=self.max_pages,
                    dtype=self.dtype, layout=self.layout)

    def _copy(self, pairs, n) -> None:
        for layer in range(self.layers):
            attn_cache_copy(self.pool[layer, 0], self.pool[layer, 1], pairs, n_copies=n, num_pages=self.num_pages,
                            page_elems=self.page_size * self.Nkv * self.D, dtype=self.dtype)

    def reserve(self, new_tokens=None, *, live_only: bool = False) -> None:
        """The rows are about to get `new_tokens` (int32 [rows] on the device; None: one each, with `live_only` one for
        each row that is not empty) more tokens: gives every row pages of its own for them and adds them to the
        lengths. Where too few pages are free nothing changes and check() raises; the rest of the step then does no
        harm (append writes nothing, attend sees the tokens from before), and once pages are free reserve can be
        called again."""
        attn_cache_grow(self.page_table, self.ref_count, self.seq_lens, new_tokens, self.new_lens, self._copies,
                        B=self.rows, max_pages=self.max_pages, num_pages=self.num_pages, page_size=self.page_size,
                        live_only=live_only)
        self._copy(self._copies, self.rows)

    def append(self, layer: int, k, v, cu_seqlens=None) -> None:
        """Writes the reserved tokens' keys and values [T, Nkv, D], packed row after row (cumulative tokens
        cu_seqlens as attn_cache_append takes them; None: one per row). Tokens of rows for which the last reserve had
        none, or was refused, are skipped. No fork comes between the two."""
        attn_cache_append(k, v, self.page_table, self.new_lens, self.pool[layer, 0], self.pool[layer, 1],
                          cu_seqlens=cu_seqlens, T=k.shape[0], B=self.rows, **self._sizes())

    def attend(self, layer: int, q, out, softmax_max=None, softmax_sum=None) -> None:
        """Attention of the newest token of each row, q and out [rows, Nq, D]."""
        attn_decode_paged(q, self.pool[layer, 0], self.pool[layer, 1], self.page_table, self.seq_lens, B=self.rows,
                          Nq=self.Nq, scale=self.scale, window_tokens=self.window_tokens, sink_tokens=self.sink_tokens,
                          workspace=self.workspace, out=out, softmax_max=softmax_max, softmax_sum=softmax_sum,
                          **self._sizes())

    def prefill(self, layer: int, q, k, v, cu_seqlens, out, softmax_max=None, softmax_sum=None) -> None:
        """Attention of whole prompts, packed row after row (q, out [T, Nq, D]; k, v [T, Nkv, D]), whose tokens
        are reserved and are the rows' first ones; their keys and values go to the cache."""
        self.append(layer, k, v, cu_seqlens)
        attn_fwd_sinks(q, k, v, cu_seqlens_q=cu_seqlens, cu_seqlens_kv=cu_seqlens, B=self.rows, Sq=q.shape[0],
                       Skv=k.shape[0], Nq=self.Nq, Nkv=self.Nkv, D=self.D, scale=self.scale,
                       window_tokens=self.window_tokens, sink_tokens=self.sink_tokens, dtype=self.dtype, layout=ATTN_TND,
                       out=out, softmax_max=softmax_max, softmax_sum=softmax_sum)

    def fork(self, src_rows) -> None:
        """Row r becomes row src_rows[r] (int32 [rows] on the device), or empty where that is negative: forks,
        beam search's reordering, and rows that are done. Shared pages are separated when a row writes."""
        attn_cache_fork(self.page_table, src_rows, self.ref_count, self.page_table, self.ref_count, rows_in=self.rows,
                        rows_out=self.rows, max_pages=self.max_pages, num_pages=self.num_pages, seq_lens=self.seq_lens,
                        seq_lens_out=self.seq_lens)

    def evict(self) -> None:
        """Frees the pages that the window has left behind."""
        attn_cache_evict(self.page_table, self.ref_count, self.seq_lens, B=self.rows, max_pages=self.max_pages,
                         num_pages=self.num_pages, page_size=self.page_size, window_tokens=self.window_tokens,
                         sink_tokens=self.sink_tokens)

    def compact(self) -> None:
        """Moves all live pages to the front of the pool: live_pages (device, [1]) of them, page x to
        page_map[x]."""
        attn_cache_compact(self.page_table, self.ref_count, self.page_table, self.ref_count, self.page_map, self._moves,
                           self.live_pages, rows=self.rows, max_pages=self.max_pages, num_pages=self.num_pages)
        self._copy(self._moves, self.num_pages // 2)

    def check(self) -> None:
        """Waits for the stream and raises what the calls since the last check recorded on the device."""
        status = attn_get_last_error()
        if status != ATTN_OK:
            raise AttnError(status, "PagedCache")
