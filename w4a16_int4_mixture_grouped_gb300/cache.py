"""A paged cache as a serving loop keeps it: one pool of pages for all layers, the sequences' tables, and the calls on
them (buffers and sequencing only; every step is a call into the CUDA library)."""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import (LATENT_DIM, MoeW4A16Error, Rotary, attention_workspace, attention_workspace_size, cache_append,
               cache_append_rotary, cache_compact, cache_copy, cache_extend, cache_fork, cache_free, cache_workspace,
               clear_device_error, get_device_error, latent_attention, paged_attention, paged_chunk_attention,
               paged_chunk_workspace, paged_chunk_workspace_size)


class PagedCache:
    """Pages of num_layers layers for max_seqs sequences of up to max_pages pages each.

    Grouped heads: pool [layers * 2, num_pages, page_size, num_heads, head_dim] (a layer's keys, then its values),
    torch.bfloat16 or torch.float8_e4m3fn with k_scale / v_scale. Latent (num_heads = head_dim = None): pool
    [layers, num_pages, page_size, 576], torch.bfloat16. `refs`, `tables` and `lens` are the sequences' state."""

    def __init__(self, num_layers: int, num_pages: int, page_size: int, max_seqs: int, max_pages: int, num_q_heads: int,
                 num_heads: Optional[int] = None, head_dim: Optional[int] = None, dtype: torch.dtype = torch.bfloat16,
                 k_scale: float = 1.0, v_scale: float = 1.0, device=None):
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.latent = num_heads is None
        if self.latent != (head_dim is None):
            raise ValueError("num_heads and head_dim go together (neither: a latent cache)")
        row = (LATENT_DIM,) if self.latent else (num_heads, head_dim)
        self.page_size, self.k_scale, self.v_scale = page_size, k_scale, v_scale
        self.pool = torch.empty((num_layers * (1 if self.latent else 2), num_pages, page_size) + row, dtype=dtype, device=dev)
        self.refs = torch.zeros(num_pages, dtype=torch.int32, device=dev)
        self.tables = torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(max_seqs, dtype=torch.int32, device=dev)
        self.ws = cache_workspace(num_pages, max_seqs, dev)
        # one for the calls on single tokens and on chunks (ordered on one stream), of the larger's size
        if row[-1] == LATENT_DIM or attention_workspace_size(num_q_heads, *row) >= paged_chunk_workspace_size(num_q_heads, *row):
            self.attn_ws = attention_workspace(max_seqs, num_q_heads, *((1, LATENT_DIM) if self.latent else row), device=dev)
        else:
            self.attn_ws = paged_chunk_workspace(num_q_heads, *row, device=dev)

    def pages(self, layer: int) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """(keys, values) of a layer; a latent cache's rows are both: (rows, None)."""
        return (self.pool[layer], None) if self.latent else (self.pool[2 * layer], self.pool[2 * layer + 1])

    def extend(self, seq_ids: torch.Tensor, counts: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Room for counts (default one) new tokens a sequence -> their first positions, -1 where there is none."""
        return cache_extend(self.refs, self.tables, self.lens, seq_ids, self.page_size, self.ws, counts=counts)

    def extend_chunk(self, seq_ids: torch.Tensor, starts: torch.Tensor,
                     num_tokens: int) -> Tuple[torch.Tensor, torch.Tensor]:
        """Room for a chunk of starts[b + 1] - starts[b] new tokens of each of the sequences -> (sequence, position) of the
        num_tokens rows: what append and DecoderLayer.forward take. Rows of no chunk, and of one that did not fit, stand at -1.
        No call takes tokens back (a length that is lowered by hand leaves pages in use): drafts that may be rejected go into a
        fork, which takes the sequence's place or is freed."""
        if seq_ids.numel() == 0:
            return tuple(torch.full((num_tokens,), -1, dtype=torch.int32, device=starts.device) for _ in range(2))
        first = self.extend(seq_ids, counts=starts[1:] - starts[:-1])
        t = torch.arange(num_tokens, dtype=torch.int32, device=starts.device)
        b = torch.searchsorted(starts[1:], t, right=True).clamp_(max=seq_ids.numel() - 1)
        at = t - starts[b]
        there = (at >= 0) & (t < starts[-1]) & (first[b] >= 0)
        return seq_ids[b], torch.where(there, first[b] + at, torch.full_like(at, -1))

    def append(self, layer: int, k: torch.Tensor, v: Optional[torch.Tensor], seq_ids: torch.Tensor,
               positions: torch.Tensor) -> None:
        kp, vp = self.pages(layer)
        cache_append(k, kp, self.tables, seq_ids, positions, self.ws, v=v, v_pages=vp, k_scale=self.k_scale,
                     v_scale=self.v_scale)

    def append_rotary(self, layer: int, q: Optional[torch.Tensor], k: torch.Tensor, v: Optional[torch.Tensor],
                      seq_ids: torch.Tensor, positions: torch.Tensor, rotary: Rotary) -> Optional[torch.Tensor]:
        """append with the keys turned by their positions -> the queries turned by them."""
        kp, vp = self.pages(layer)
        return cache_append_rotary(q, k, kp, self.tables, seq_ids, positions, rotary, self.ws, v=v, v_pages=vp,
                                   k_scale=self.k_scale, v_scale=self.v_scale)

    def attend(self, layer: int, q: torch.Tensor, seq_ids: torch.Tensor, scale: float, window: int = 0) -> torch.Tensor:
        """Attention of one new token (already appended) of each of the sequences."""
        kp, vp = self.pages(layer)
        if self.latent:
            return latent_attention(q, kp, self.tables, self.lens, self.attn_ws, scale, window=window, seq_ids=seq_ids)[0]
        return paged_attention(q, kp, vp, self.tables, self.lens, self.attn_ws, scale=scale, window=window,
                               k_scale=self.k_scale, v_scale=self.v_scale, seq_ids=seq_ids)[0]

    def attend_chunk(self, layer: int, q: torch.Tensor, starts: torch.Tensor, seq_ids: torch.Tensor, scale: float,
                     window: int = 0, positions: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Causal attention of a chunk of new tokens (already appended) of each of the sequences, grouped heads: rows
        starts[b] .. starts[b + 1] - 1 are sequence seq_ids[b]'s last tokens. Rows of no chunk give zeros, and so do, given
        extend_chunk's positions, the rows of a chunk that did not fit: without them those would be taken for the last tokens
        that the sequence has."""
        if self.latent:
            raise ValueError("a latent cache is attended one token at a time")
        kp, vp = self.pages(layer)
        return paged_chunk_attention(q, starts, kp, vp, self.tables, self.lens, self.attn_ws, scale=scale, window=window,
                                     k_scale=self.k_scale, v_scale=self.v_scale, seq_ids=seq_ids,
                                     out=torch.zeros(q.shape, dtype=torch.bfloat16, device=q.device), positions=positions)[0]

    def fork(self, parents: torch.Tensor, children: torch.Tensor) -> None:
        cache_fork(self.pool, self.refs, self.tables, self.lens, parents, children, self.page_size, self.ws)

    def free(self, seq_ids: torch.Tensor, keep: Optional[torch.Tensor] = None) -> None:
        cache_free(self.refs, self.tables, self.lens, seq_ids, self.page_size, self.ws, keep=keep)

    def copy(self, src: torch.Tensor, dst: torch.Tensor) -> None:
        cache_copy(self.pool, src, dst, self.ws)

    def compact(self) -> torch.Tensor:
        """Pages in use to the front of the pool -> their number [1]."""
        return cache_compact(self.pool, self.refs, self.tables, self.ws, refs_out=self.refs, tables_out=self.tables)[3]

    def check(self) -> None:
        """Synchronises; raises (and clears) what the calls so far recorded: no free page, an id out of range."""
        for ws in (self.ws, self.attn_ws):
            code = get_device_error(ws)
            if code:
                clear_device_error(ws)
                raise MoeW4A16Error(code, "PagedCache")
