"""A sparse-attention layer's decode step: the indexer selects, the layer's keys
and values are appended, and the rows attend.

``DecodeAttention`` owns what a serving loop keeps between steps besides the
indexer's own state: the paged key/value cache (same pages and slots as the
indexer's cache; in 16 bits or in 4), the angle table and the workspaces.  ``step`` runs indexer,
append and attention over the selected keys on the current stream;
``dense_step`` runs append and attention over all keys, behind a prefix that
the batch may share, for layers without an indexer.  Both can be captured into
a CUDA graph.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import dsa
from .step import DecodeIndexer, StepOutput


def angle_table(max_pos: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """FP32 [max_pos, rot_dim]: cosines, then sines, of position * base^(-2i / rot_dim)
    (angles in FP64, so that far positions keep theirs)."""
    freq = base ** (-torch.arange(0, rot_dim, 2, device=device, dtype=torch.float64) / rot_dim)
    angle = torch.arange(max_pos, device=device, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).to(torch.float32)


class DecodeAttention:
    def __init__(self, indexer: DecodeIndexer, heads: int, kv_heads: int, dim: int, cos_sin: torch.Tensor,
                 max_rows: int, max_query_len: int, dtype: torch.dtype = torch.bfloat16, interleaved: bool = False,
                 scale: Optional[float] = None, kv_format: Optional[str] = None, k_scale: float = 1.0,
                 v_scale: float = 1.0):
        """kv_format: None for a cache of ``dtype``, "nvfp4" for one in 4 bits (E2M1 codes with an E4M3 scale per 16
        columns) whose FP32 scales are ``k_scale`` and ``v_scale``; ``dtype`` is that of q, k, v and the output."""
        if kv_format not in (None, "nvfp4"):
            raise ValueError(f"unknown kv_format {kv_format!r}; expected None or 'nvfp4'")
        self.indexer = indexer
        dev = indexer.device
        pages = max(1, indexer.num_pages)
        self.dim, self.dtype, self.kv_format = int(dim), dtype, kv_format
        if kv_format is None:
            shape = (pages, dsa.PAGE_TOKENS, kv_heads, dim)
            self.k_cache = torch.zeros(shape, dtype=dtype, device=dev)
            self.v_cache = torch.zeros(shape, dtype=dtype, device=dev)
        else:
            self.kv_cache = dsa.new_kv_cache_fp4(pages, kv_heads, dim, dev)
            self.kv_scales = dict(k_scale=float(k_scale), v_scale=float(v_scale))
        self.cos_sin = cos_sin.to(dev, torch.float32).contiguous()
        self.interleaved, self.scale, self.max_query_len = bool(interleaved), scale, int(max_query_len)
        requests = indexer.block_table.shape[0]
        sizes = dsa.attend_workspace_size if kv_format is None else dsa.attend_workspace_size_fp4
        size = max(sizes(max_rows, requests, heads, kv_heads, dim, self.max_query_len),
                   sizes(max_rows, requests, heads, kv_heads, dim, 1, max(indexer.k, 1)))
        # (not the indexer's, which has to stay clear; this one needs no clearing)
        self.workspace = torch.empty(max(size, 256), dtype=torch.uint8, device=dev)

    def append(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, positions: torch.Tensor,
               q: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
        """Keys and values into their slots, keys (and queries) rotated; returns the rotated queries."""
        if self.kv_format is not None:
            return dsa.kv_append_fp4(k, v, slots, self.kv_cache, positions, self.cos_sin, q=q,
                                     interleaved=self.interleaved, status=self.indexer.status, **self.kv_scales)
        return dsa.kv_append(k, v, slots, self.k_cache, self.v_cache, positions, self.cos_sin, q=q,
                             interleaved=self.interleaved, status=self.indexer.status)

    def read(self, slots: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
        """The keys and values [n, kv_heads, dim] that a 4-bit cache holds in slots (int64 [n], -1: zeros), as a later
        chunk of a prompt needs them."""
        if self.kv_format is None:
            raise ValueError("a 16-bit cache is read as it is: k_cache and v_cache")
        return dsa.kv_read_fp4(slots, self.kv_cache, self.dim, self.dtype, status=self.indexer.status,
                               **self.kv_scales)

    def _table(self, starts: torch.Tensor) -> torch.Tensor:
        """The block table of the step's requests, the first of the indexer's."""
        table, requests = self.indexer.block_table, starts.numel() - 1
        return table if table.shape[0] == requests else table[:requests]

    def step(self, iq: torch.Tensor, wv: torch.Tensor, ikeys: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
             v: torch.Tensor, slots: torch.Tensor, positions: torch.Tensor, seq_lens: torch.Tensor,
             query_lens: torch.Tensor) -> Tuple[torch.Tensor, StepOutput]:
        """iq [rows, 32, 128], wv [rows, 32], ikeys [rows, 128]: the indexer's projections; q [rows, heads, dim],
        k and v [rows, kv_heads, dim]: the layer's; slots and positions int64 [rows] (slot -1: padding); a request for
        each of the block table's rows or of its first.
        Returns (attention output [rows, heads, dim], the indexer's step)."""
        chosen = self.indexer.step(iq, wv, ikeys, slots, seq_lens, query_lens, self.max_query_len)
        q = self.append(k, v, slots, positions, q)
        if self.kv_format is not None:
            out, _ = dsa.attend_selected_fp4(q, self.kv_cache, self._table(chosen.starts), chosen.starts,
                                             chosen.row_ends, chosen.topk, scale=self.scale, workspace=self.workspace,
                                             status=self.indexer.status, **self.kv_scales)
            return out, chosen
        out, _ = dsa.attend_selected(q, self.k_cache, self.v_cache, self._table(chosen.starts), chosen.starts,
                                     chosen.row_ends, chosen.topk, scale=self.scale, workspace=self.workspace,
                                     status=self.indexer.status)
        return out, chosen

    def dense_step(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                   positions: torch.Tensor, starts: torch.Tensor, row_ends: torch.Tensor,
                   prefix_pages: Optional[torch.Tensor] = None, prefix_len: int = 0) -> torch.Tensor:
        """Append, then attention over the shared prefix (16-bit caches; requests of a 4-bit cache list its pages in
        their own tables) and all own keys below ``row_ends``.  The layer's ``max_query_len`` and the block table's
        width go into the call as they are: a 4-bit layer of short requests is faster with both no larger than it
        needs."""
        if self.kv_format is not None:
            if prefix_len != 0:
                raise ValueError("a shared prefix is read from a 16-bit cache only")
            q = self.append(k, v, slots, positions, q)
            out, _ = dsa.attend_paged_fp4(q, self.kv_cache, self._table(starts), starts, row_ends, self.max_query_len,
                                          scale=self.scale, workspace=self.workspace, status=self.indexer.status,
                                          **self.kv_scales)
            return out
        q = self.append(k, v, slots, positions, q)
        out, _ = dsa.attend_paged(q, self.k_cache, self.v_cache, self._table(starts), starts, row_ends,
                                  self.max_query_len, prefix_pages=prefix_pages, prefix_len=prefix_len,
                                  scale=self.scale, workspace=self.workspace, status=self.indexer.status)
        return out
