"""Host-side planning of a mixed prefill/decode batch.

A serving step gathers new tokens from many requests; each request owns one
running state in a pool (its slot).  Requests with exactly one new token are
routed to the decode kernel, the others are packed as variable-length prefill
chunks ("MiniMax-01技术报告解读", §3.3 item 2: prefill and decode on separate
streams, length-1 tokens through the decode kernel).  `plan_batch` decides the
row order of the packed batch that `mixed_step` expects -- prefill chunks
first, then one row per decode token -- and builds the index arrays.  It does
no GPU work; placing each request's q, k, v rows at `row_offset` is the
caller's part.

`PagePool` keeps the page numbers of the softmax layers' key/value caches: which
pages a request owns or shares with its forks, which are free, and which copies
the caches need (`cache_copy_pages`) before the next step reads or writes them.
One pool serves every layer, whose cache tensors share its numbering.  It does
no GPU work either.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np


@dataclass
class BatchPlan:
    prefill_ids: np.ndarray    # request indices packed as prefill chunks, in row order
    decode_ids: np.ndarray     # request indices served by the decode kernel, in row order
    row_offset: np.ndarray     # [n_requests] first row of each request (-1: no new tokens)
    cu_seqlens: np.ndarray     # int32 [n_prefill + 1] over the prefill rows
    prefill_slots: np.ndarray  # int32 [n_prefill]
    decode_slots: np.ndarray   # int32 [n_decode]
    prefill_tokens: int
    max_seqlen: int

    @property
    def total_rows(self) -> int:
        return self.prefill_tokens + len(self.decode_ids)


def plan_batch(lengths, slots) -> BatchPlan:
    """lengths[i]: new tokens of request i (>= 0); slots[i]: its state slot.
    Requests with no new tokens take no rows; one slot may serve one request."""
    lengths = np.asarray(lengths, dtype=np.int64)
    slots = np.asarray(slots, dtype=np.int64)
    if lengths.shape != slots.shape or lengths.ndim != 1:
        raise ValueError("lengths and slots must be 1-D and of equal length")
    if (lengths < 0).any():
        raise ValueError("negative length")
    active = lengths > 0
    if len(np.unique(slots[active])) != int(active.sum()):
        raise ValueError("two requests of one batch share a state slot")
    prefill_ids = np.nonzero(lengths > 1)[0]
    decode_ids = np.nonzero(lengths == 1)[0]
    cu = np.zeros(len(prefill_ids) + 1, dtype=np.int64)
    np.cumsum(lengths[prefill_ids], out=cu[1:])
    prefill_tokens = int(cu[-1])
    if prefill_tokens + len(decode_ids) > 0x7FFFFFFF:
        raise ValueError("batch too large")
    row_offset = np.full(len(lengths), -1, dtype=np.int64)
    row_offset[prefill_ids] = cu[:-1]
    row_offset[decode_ids] = prefill_tokens + np.arange(len(decode_ids))
    return BatchPlan(prefill_ids=prefill_ids, decode_ids=decode_ids, row_offset=row_offset,
                     cu_seqlens=cu.astype(np.int32), prefill_slots=slots[prefill_ids].astype(np.int32),
                     decode_slots=slots[decode_ids].astype(np.int32), prefill_tokens=prefill_tokens,
                     max_seqlen=int(lengths[prefill_ids].max()) if len(prefill_ids) else 0)


class PoolExhausted(RuntimeError):
    """More pages are asked for than are free."""


class PagePool:
    """Page numbers of paged key/value caches [n_pages, Hkv, page_size, d].

    A request's tokens lie in its pages in order.  A fork shares all pages of
    its parent; whichever of them writes to a shared, ragged last page first
    gets a copy of it (`reserve`).  Copies collect until `take_copies`, whose
    arrays go to one `cache_copy_pages` call per layer, in front of the step;
    until then no page that a collected copy reads or writes is given out
    again, so a call never names a page as source and destination.
    """

    def __init__(self, n_pages: int, page_size: int):
        if n_pages <= 0 or page_size not in (16, 32, 64, 128):
            raise ValueError("n_pages must be positive, page_size 16, 32, 64 or 128")
        self.n_pages, self.page_size = int(n_pages), int(page_size)
        self._free = list(range(self.n_pages - 1, -1, -1))   # lowest number on top
        self._refs = [0] * self.n_pages                      # requests that hold the page
        self._pages: dict[int, list[int]] = {}
        self._lens: dict[int, int] = {}
        self._copies: list[tuple[int, int]] = []
        self._held: set[int] = set()      # pages of collected copies
        self._next = 0

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def __contains__(self, request) -> bool:
        return request in self._pages

    def length(self, request: int) -> int:
        """Tokens cached for the request."""
        return self._lens[request]

    def pages(self, request: int) -> list[int]:
        return list(self._pages[request])

    def add(self) -> int:
        """A new request without tokens."""
        request, self._next = self._next, self._next + 1
        self._pages[request], self._lens[request] = [], 0
        return request

    def reserve(self, request: int, new_tokens: int) -> None:
        """Pages for new_tokens behind the request's cached ones, none of them
        shared where they will be written.  Raises PoolExhausted, changing
        nothing, when too few are free."""
        if new_tokens < 0:
            raise ValueError("negative number of tokens")
        if new_tokens == 0:
            return
        pages, n = self._pages[request], self._lens[request]
        first = n // self.page_size                       # page of the first new token
        last = -(-(n + new_tokens) // self.page_size)
        shared = [i for i in range(first, min(last, len(pages))) if self._refs[pages[i]] > 1]
        need = max(0, last - len(pages)) + len(shared)
        if need > len(self._free):
            raise PoolExhausted(f"{need} pages needed, {len(self._free)} free")
        for i in shared:
            page = self._take()
            if i * self.page_size < n:                    # it holds tokens: the ragged page
                # (a page that a collected copy is still to fill: that copy's source)
                src = next((s for s, d in self._copies if d == pages[i]), pages[i])
                self._copies.append((src, page))
                self._held.update((src, page))
            self._drop(pages[i])
            pages[i] = page
        while len(pages) < last:
            pages.append(self._take())

    def advance(self, request: int, tokens: int) -> None:
        """The step has written `tokens` new tokens of the request."""
        n = self._lens[request] + tokens
        if tokens < 0 or n > len(self._pages[request]) * self.page_size:
            raise ValueError("more tokens than were reserved")
        self._lens[request] = n

    def fork(self, request: int) -> int:
        """A new request with the same tokens, sharing all pages."""
        child = self.add()
        keep = -(-self._lens[request] // self.page_size)  # reserved pages without tokens stay the parent's
        self._pages[child], self._lens[child] = self._pages[request][:keep], self._lens[request]
        for page in self._pages[child]:
            self._refs[page] += 1
        return child

    def free(self, request: int) -> None:
        """Give back the request's pages (those that no fork holds)."""
        for page in self._pages.pop(request):
            self._drop(page)
        del self._lens[request]

    def take_copies(self):
        """(src, dst) int32 arrays of the copies collected so far, for
        cache_copy_pages on every layer's cache; clears them."""
        pairs = np.array(self._copies, dtype=np.int32).reshape(-1, 2)
        self._copies = []
        held, self._held = self._held, set()
        for page in sorted(held, reverse=True):
            if self._refs[page] == 0:
                self._free.append(page)
        return np.ascontiguousarray(pairs[:, 0]), np.ascontiguousarray(pairs[:, 1])

    def compact(self):
        """Move the pages in use to the lowest numbers, tables included; (src,
        dst) of the copies as from `take_copies`.  Refused while copies are
        collected."""
        if self._copies:
            raise RuntimeError("take the collected copies first")
        used = [p for p in range(self.n_pages) if self._refs[p]]
        moves = {}
        holes = [p for p in range(len(used)) if not self._refs[p]]
        for src, dst in zip(reversed(used), holes):
            if src < dst:
                break
            moves[src] = dst
        for src, dst in moves.items():
            self._refs[dst], self._refs[src] = self._refs[src], 0
        for pages in self._pages.values():
            pages[:] = [moves.get(p, p) for p in pages]
        self._free = [p for p in range(self.n_pages - 1, -1, -1) if not self._refs[p]]
        pairs = np.array(list(moves.items()), dtype=np.int32).reshape(-1, 2)
        return np.ascontiguousarray(pairs[:, 0]), np.ascontiguousarray(pairs[:, 1])

    def table(self, requests, max_pages: int | None = None) -> np.ndarray:
        """int32 [requests, max_pages] page table; None in `requests` is a row
        without a request, entries behind a request's pages are 0."""
        rows = [[] if r is None else self._pages[r] for r in requests]
        width = max([len(x) for x in rows] + [1])
        if max_pages is None:
            max_pages = width
        elif max_pages < width:
            raise ValueError(f"a request has {width} pages, the table {max_pages}")
        out = np.zeros((len(rows), max_pages), dtype=np.int32)
        for i, x in enumerate(rows):
            out[i, :len(x)] = x
        return out

    def lengths(self, requests) -> np.ndarray:
        """int32 cached tokens, -1 for a row without a request."""
        return np.array([-1 if r is None else self._lens[r] for r in requests], dtype=np.int32)

    def _take(self) -> int:
        page = self._free.pop()
        self._refs[page] = 1
        return page

    def _drop(self, page: int) -> None:
        self._refs[page] -= 1
        if self._refs[page] == 0 and page not in self._held:
            self._free.append(page)
