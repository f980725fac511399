"""A persistent cache of documents in 8 bits: pages of quantised rows on the device, and on the host which
document has which pages.

The kernels are ``kalm_cache_write`` and ``kalm_cache_read`` (and ``kalm_merged_attention_cache``, which reads a
scorer's cached cross K/V); this class hands out pages, so that no two rows share a place, and builds the page
tables that the calls take.  A row is one pooled vector ("KaLM-Reranker-V1-Nano - MLX (Apple Silicon)", "What this
is": each passage is encoded and chunk-pooled once) or whatever a caller keeps per pooled vector, e.g. its cross
K/V of every layer: 1 + 1/32 bytes a value.

Calls are asynchronous on the current stream.  Pages that ``drop`` frees are handed out again at once, so
reads and writes of one cache belong on one stream (or on streams that the caller orders).
"""
from __future__ import annotations

import dataclasses
from typing import Hashable, Optional, Sequence

import numpy as np
import torch

from . import CACHE_GROUP, kalm_cache_read, kalm_cache_write


@dataclasses.dataclass
class CacheView:
    """Some documents of a cache, as the calls on it take them (device tensors, in the order asked for)."""
    page_table: torch.Tensor  # int32 [n][pages], -1 past a document's last page
    row_off: torch.Tensor     # int64 [n + 1]: packed rows of each document
    rows: list                # rows of each document (host)

    @property
    def total_rows(self) -> int:
        return sum(self.rows)


class DocumentCache:
    """``n_pages`` pages of ``page_rows`` rows of ``width`` values (a multiple of 32).  ``layout`` says what a row's
    columns are, for callers to compare (the cache itself does not read it)."""

    def __init__(self, n_pages: int, width: int, page_rows: int = 64, device="cuda", layout: Hashable = None):
        if n_pages < 0 or width <= 0 or width % CACHE_GROUP:
            raise ValueError(f"DocumentCache: n_pages={n_pages}, width={width} (a positive multiple of {CACHE_GROUP})")
        if page_rows not in (8, 16, 32, 64, 128, 256, 512, 1024):
            raise ValueError(f"DocumentCache: page_rows={page_rows} is not a power of two in [8, 1024]")
        self.n_pages, self.width, self.page_rows, self.device = n_pages, width, page_rows, torch.device(device)
        self.layout = layout
        self.codes = torch.zeros(n_pages * page_rows, width, dtype=torch.uint8, device=device)
        self.scales = torch.zeros(n_pages * page_rows, width // CACHE_GROUP, dtype=torch.uint8, device=device)
        self._free = list(range(n_pages - 1, -1, -1))  # taken from the end: page 0 first
        self._docs: dict = {}                          # key -> (pages, rows)

    def __contains__(self, key: Hashable) -> bool:
        return key in self._docs

    def __len__(self) -> int:
        return len(self._docs)

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def rows(self, key: Hashable) -> int:
        return self._docs[key][1]

    # ------------------------------------------------------------------ writing
    def put(self, keys: Sequence[Hashable], rows: Sequence[int], src: torch.Tensor) -> None:
        """New documents: ``src`` holds their rows packed one document after another (bf16 [sum(rows)][width])."""
        self._check_new(keys)
        self._write(keys, rows, src)

    def check_put(self, keys: Sequence[Hashable], rows: Sequence[int]) -> None:
        """Raise what ``put`` of these documents would raise for their keys, row counts and pages."""
        self._check_new(keys)
        self._plan(keys, rows)

    def _check_new(self, keys) -> None:
        for k in keys:
            if k in self._docs:
                raise KeyError(f"document {k!r} is cached already: drop it first, or append to it")

    def append(self, keys: Sequence[Hashable], rows: Sequence[int], src: torch.Tensor) -> None:
        """More rows of cached documents (down to a single row), packed as for ``put``."""
        for k in keys:
            if k not in self._docs:
                raise KeyError(f"document {k!r} is not cached")
        self._write(keys, rows, src)

    def _plan(self, keys, rows) -> tuple:
        """(row counts, (pages, rows) held, new pages needed) of each document of a write."""
        rows = [int(r) for r in rows]
        if len(rows) != len(keys) or any(r < 0 for r in rows):
            raise ValueError(f"{len(keys)} documents, row counts {rows}")
        if len(set(keys)) != len(keys):
            raise ValueError("a document is named twice in one write")
        old = [self._docs.get(k, ([], 0)) for k in keys]
        need = [-(-(o[1] + r) // self.page_rows) - len(o[0]) for o, r in zip(old, rows)]
        if sum(need) > len(self._free):
            raise MemoryError(f"the cache has {len(self._free)} free pages, {sum(need)} are needed")
        return rows, old, need

    def _write(self, keys, rows, src) -> None:
        rows, old, need = self._plan(keys, rows)
        if src.dim() != 2 or tuple(src.shape) != (sum(rows), self.width):
            raise ValueError(f"src has shape {tuple(src.shape)}, expected ({sum(rows)}, {self.width})")
        taken = [self._free[len(self._free) - 1 - i] for i in range(sum(need))]
        pages, at = [], 0
        for o, n in zip(old, need):
            pages.append(o[0] + taken[at:at + n])
            at += n
        if sum(rows):
            first = np.array([o[1] for o in old], dtype=np.int32)
            kalm_cache_write(src, self._device(_offsets(rows)), self._device(_table(pages)), self.page_rows, self.codes,
                             self.scales, first_row=self._device(first) if first.any() else None)
        # the call was accepted: the documents have their pages
        if taken:
            del self._free[-len(taken):]
        for k, p, o, r in zip(keys, pages, old, rows):
            self._docs[k] = (p, o[1] + r)

    def drop(self, keys: Sequence[Hashable]) -> None:
        """Forget documents; their pages are free at once."""
        if len(set(keys)) != len(keys):
            raise ValueError("a document is named twice")
        for k in keys:
            if k not in self._docs:
                raise KeyError(f"document {k!r} is not cached")
        for k in keys:
            self._free.extend(reversed(self._docs.pop(k)[0]))

    # ------------------------------------------------------------------ reading
    def view(self, keys: Sequence[Hashable]) -> CacheView:
        """The page table and row offsets of some documents (a document may be named more than once)."""
        docs = [self._docs[k] for k in keys]
        rows = [r for _, r in docs]
        return CacheView(self._device(_table([p for p, _ in docs])), self._device(_offsets(rows)), rows)

    def get(self, keys: Sequence[Hashable], out: Optional[torch.Tensor] = None) -> tuple:
        """(rows, offsets): the documents' rows packed one after another, bf16, as stored."""
        v = self.view(keys)
        if out is None:
            out = torch.empty(v.total_rows, self.width, dtype=torch.bfloat16, device=self.device)
        elif out.dim() != 2 or tuple(out.shape) != (v.total_rows, self.width):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected ({v.total_rows}, {self.width})")
        if v.total_rows:
            kalm_cache_read(self.codes, self.scales, v.row_off, v.page_table, self.page_rows, out)
        return out, v.row_off

    def _device(self, a: np.ndarray) -> torch.Tensor:
        return torch.from_numpy(a).to(self.device)


def _offsets(rows) -> np.ndarray:
    off = np.zeros(len(rows) + 1, dtype=np.int64)
    np.cumsum(rows, out=off[1:])
    return off


def _table(pages) -> np.ndarray:
    table = np.full((len(pages), max((len(p) for p in pages), default=0)), -1, dtype=np.int32)
    for d, p in enumerate(pages):
        table[d, :len(p)] = p
    return table
