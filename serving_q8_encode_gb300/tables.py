"""Block tables, lengths and free pages of the slots that a server fills, kept and changed on the GPU."""
from __future__ import annotations

from typing import NamedTuple

import torch

from .pages import _ext


class Plan(NamedTuple):
    """What a step's calls take. starts: int32 [A + 1], the packed rows of each slot. before, after: int32 [A], its length
    before the step (append's lens) and with the new tokens (attend's, attend_rows's and gather's), -1 for a slot that takes
    no part. slots: int64 [n_rows], page id * page_tokens + place in the page; positions: int64 [n_rows], place in the
    sequence; -1 in both for a row that is not appended."""
    starts: torch.Tensor
    before: torch.Tensor
    after: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor


class PageTable:
    """Which pages of a PageCache each slot's sequence has, and which are free.

    n_seqs slots of up to max_pages pages each, over n_pages pages of page_tokens tokens. window, sinks: as the attention
    that reads the pages takes them; pages that it can no longer see are given back as the sequences grow.

    Device tensors: block_table int32 [A][max_pages] (-1: none) and lens int32 [A] (-1: idle), as the cache's calls take
    them; first int32 [A], ring int32 [n_pages], counts int64 [2]: the rest of the state (see polykv_page_tables). plan and
    cut change them on ``stream``, or on the current stream of their device; calls on one table must be ordered on the GPU.
    Nothing is read back to the host: a captured graph follows the tensors' contents."""

    def __init__(self, n_seqs: int, max_pages: int, n_pages: int, page_tokens: int = 32, window: int = 0, sinks: int = 0,
                 device="cuda"):
        if n_seqs < 1 or max_pages < 1 or n_pages < 1:
            raise ValueError("n_seqs, max_pages and n_pages must be at least 1")
        if page_tokens not in (16, 32, 64, 128):
            raise ValueError(f"page_tokens must be 16, 32, 64 or 128, got {page_tokens}")
        if not 0 <= window < 1 << 31 or not 0 <= sinks < 1 << 31:
            raise ValueError(f"window ({window}) and sinks ({sinks}) must be between 0 and 2^31 - 1")
        self.n_seqs, self.max_pages, self.n_pages, self.page_tokens = n_seqs, max_pages, n_pages, page_tokens
        self.window, self.sinks = window, sinks
        ints = dict(dtype=torch.int32, device=device)
        self.block_table = torch.full((n_seqs, max_pages), -1, **ints)
        self.lens = torch.full((n_seqs,), -1, **ints)
        self.first = torch.full((n_seqs,), -(-sinks // page_tokens), **ints)
        self.ring = torch.arange(n_pages, **ints)
        self.counts = torch.tensor([0, n_pages], dtype=torch.int64, device=device)
        self.device = self.block_table.device
        self._arrivals = torch.zeros(1, **ints)
        self._status = torch.zeros(1, **ints)
        self._t = _ext.tables(self.block_table, self.lens, self.first, self.ring, self.counts, self._arrivals, self._status,
                              page_tokens, window, sinks)

    def _on(self, stream):
        if stream.device != self.device:
            raise ValueError(f"stream is on {stream.device}, the tables on {self.device}")
        return torch.cuda.stream(stream)

    def plan(self, new, n_rows: int, stream=None) -> Plan:
        """A step that appends new[s] tokens (device int32 [A]; negative counts as 0) to each slot, in n_rows packed rows; an
        idle slot begins a sequence. Slots are served in order: one is granted if its new pages are free, its table has room
        and its rows end within n_rows; one that needs pages is not once one before it was refused for lack of pages. A slot
        that is not granted keeps its state and takes no part (-1 in ``before`` and ``after``), its rows stay in their places."""
        if stream is not None:
            with self._on(stream):
                return self.plan(new, n_rows)
        return Plan(*_ext.tables_plan(self._t, new, n_rows))

    def cut(self, keep, stream=None) -> None:
        """Each slot keeps the first keep[s] tokens of its sequence (device int32 [A]; as many as it has if that is fewer):
        drafted tokens that were rejected. Negative: the sequence ends, the slot is idle. Their pages are free for the next
        plan. With a window a sequence can be cut to its length before the last plan, not further."""
        if stream is not None:
            with self._on(stream):
                return self.cut(keep)
        _ext.tables_cut(self._t, keep)

    def restore(self, block_table, lens, first, ring, counts) -> None:
        """Takes a saved state: copies of the tensors of these names."""
        for name, t in dict(block_table=block_table, lens=lens, first=first, ring=ring, counts=counts).items():
            mine = getattr(self, name)
            if tuple(t.shape) != tuple(mine.shape) or t.dtype != mine.dtype:
                raise ValueError(f"{name} must be {mine.dtype} {tuple(mine.shape)}, got {t.dtype} {tuple(t.shape)}")
        for name, t in dict(block_table=block_table, lens=lens, first=first, ring=ring, counts=counts).items():
            getattr(self, name).copy_(t)

    def status(self, stream=None) -> int:
        """Raises PolyKVError (E_STATE) if a plan or a cut met a page id outside the pages, a length beyond the table, or more
        rows than n_rows or than the table holds, since the last call (synchronises)."""
        if stream is not None:
            with self._on(stream):
                return _ext.tables_status(self._t)
        return _ext.tables_status(self._t)
