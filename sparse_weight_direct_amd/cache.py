"""The pages of a cache that several attention layers share, counted on the host.

One tensor holds every layer's keys and values, (2 * layers, pages, values a page), so that one
cache_copy moves a page in all of them.  A sequence is a list of pages and a length; sequences may share
pages (fork), and a page that a sequence is about to write is its own: extend() copies a shared one first.
The counting is the host's alone (nothing is read back); copies and tables are made on the current
stream, in order with the calls that use them.  Each list that goes to the GPU (extend: a table and a past, and the pages to copy where
there are any) is copied from pageable memory, so the host waits there until the stream has come to it, and none of it can be captured
into a graph: a graph's steps advance a past of their own, over a table that was extended before.
"""
from __future__ import annotations

import torch

from .attention import cache_copy


class PagePool:
    """`pages` pages of `page_size` positions (16, 32, 64, 128 or 256) for `layers` layers of `heads` heads of `dims` dims."""

    def __init__(self, layers: int, pages: int, heads: int, dims: int, *, page_size: int = 64, dtype=torch.float32, device="cuda"):
        if min(layers, pages, heads, dims) < 1 or page_size not in (16, 32, 64, 128, 256):
            raise ValueError("layers, pages, heads, dims >= 1 and a page_size of 16, 32, 64, 128 or 256")
        self.layers, self.pages, self.heads, self.dims, self.page_size = layers, pages, heads, dims, page_size
        self.pool = torch.zeros(2 * layers, pages, heads * page_size * dims, dtype=dtype, device=device)
        self._free = list(range(pages - 1, -1, -1))  # the lowest on top
        self._users = [0] * pages
        self._pages: dict[int, list[int]] = {}
        self._length: dict[int, int] = {}
        self._next = 0

    def k_pages(self, layer: int):
        return self.pool[2 * layer].view(self.pages, self.heads, self.page_size, self.dims)

    def v_pages(self, layer: int):
        return self.pool[2 * layer + 1].view(self.pages, self.heads, self.dims, self.page_size)

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def length(self, sequence: int) -> int:
        return self._length[sequence]

    def add(self) -> int:
        """A new, empty sequence."""
        s, self._next = self._next, self._next + 1
        self._pages[s], self._length[s] = [], 0
        return s

    def fork(self, sequence: int) -> int:
        """A new sequence with the same positions.  No page is copied before one of the two is extended."""
        pages, length = list(self._pages[sequence]), self._length[sequence]
        s = self.add()
        for p in pages:
            if p >= 0:
                self._users[p] += 1
        self._pages[s], self._length[s] = pages, length
        return s

    def _drop(self, page: int) -> None:
        self._users[page] -= 1
        if self._users[page] == 0:
            self._free.append(page)

    def free(self, sequence: int) -> None:
        """Gives the sequence's pages back (those that no other has)."""
        pages = self._pages.pop(sequence)
        del self._length[sequence]
        for p in pages:
            if p >= 0:
                self._drop(p)

    def extend(self, sequences, lengths, *, width: int | None = None):
        """Room for lengths[i] more positions of sequences[i]; returns (table, past), int32 on the pool's device, for the calls
        that write them.  The sequences' lengths grow at once: if a call that was to write them is refused, truncate() takes the
        positions back, or the next call attends to what was never written.  MemoryError, and nothing changed, where there are too
        few pages.  width: of the table (default: as few pages as hold the longest)."""
        sequences, lengths = list(sequences), [int(n) for n in lengths]
        if len(sequences) != len(lengths) or len(set(sequences)) != len(sequences):
            raise ValueError("a length for each sequence, and each sequence once")
        if any(n < 0 for n in lengths):
            raise ValueError("a length is negative")
        P = self.page_size
        wanted, users = [], list(self._users)
        for s, n in zip(sequences, lengths):
            pages, old = self._pages[s], self._length[s]
            last = n > 0 and old % P != 0 and users[pages[-1]] > 1  # its half filled page is another's too
            if last:
                users[pages[-1]] -= 1
            wanted.append((last, -(-(old + n) // P) - len(pages)))
        need = sum(last + new for last, new in wanted)
        if need > len(self._free):
            raise MemoryError(f"{need} pages wanted, {len(self._free)} free")
        longest = max((len(self._pages[s]) + new for s, (_, new) in zip(sequences, wanted)), default=0)
        if width is None:
            width = max(1, longest)
        elif width < longest:
            raise ValueError(f"a table of {width} pages where a sequence has {longest}")
        past, copies = [], []
        for s, n, (last, new) in zip(sequences, lengths, wanted):
            pages, old = self._pages[s], self._length[s]
            past.append(old)
            if last:
                fresh = self._take()
                copies.append((pages[-1], fresh))
                self._drop(pages[-1])
                pages[-1] = fresh
            pages += [self._take() for _ in range(new)]
            self._length[s] = old + n
        self._copy(copies)
        return self.table(sequences, width=width), self._ints(past)

    def truncate(self, sequence: int, length: int) -> None:
        """Takes back the sequence's positions from `length` on, and gives back the pages that only they used."""
        pages, P = self._pages[sequence], self.page_size
        keep = -(-length // P)
        if not 0 <= length <= self._length[sequence] or (length % P and pages[keep - 1] < 0):
            raise ValueError(f"a length of {length} where the sequence has {self._length[sequence]}, or inside a page that forget() gave back")
        for p in pages[keep:]:
            if p >= 0:
                self._drop(p)
        del pages[keep:]
        self._length[sequence] = length

    def _take(self) -> int:
        p = self._free.pop()
        self._users[p] = 1
        return p

    def _ints(self, v):
        return torch.tensor(v, dtype=torch.int32).to(self.pool.device)

    def _copy(self, pairs) -> None:
        if pairs:
            both = self._ints([list(x) for x in zip(*pairs)])
            cache_copy(self.pool, both[0], both[1])

    def table(self, sequences, *, width: int | None = None):
        """(len(sequences), width) int32 on the pool's device: each sequence's pages, then -1."""
        lists = [self._pages[s] for s in sequences]
        longest = max((len(p) for p in lists), default=0)
        width = max(1, longest) if width is None else width
        if width < longest:
            raise ValueError(f"a table of {width} pages where a sequence has {longest}")
        return self._ints([p + [-1] * (width - len(p)) for p in lists]).view(len(lists), width)

    def forget(self, sequence: int, before: int) -> None:
        """Gives back the pages of positions that all lie before `before` (a window has passed them): their entries in
        tables are -1 from now on, and nobody sees them."""
        pages = self._pages[sequence]
        for i in range(min(before, self._length[sequence]) // self.page_size):
            if pages[i] >= 0:
                self._drop(pages[i])
                pages[i] = -1

    def compact(self) -> int:
        """Moves the pages in use to the pool's beginning; returns how many they are.  Tables made before are no longer valid."""
        used = self.pages - len(self._free)
        holes = sorted(p for p in self._free if p < used)
        high = [p for p in range(used, self.pages) if self._users[p]]
        to = dict(zip(high, holes))
        self._copy(list(to.items()))
        for pages in self._pages.values():
            pages[:] = [to.get(p, p) for p in pages]
        for a, b in to.items():
            self._users[b], self._users[a] = self._users[a], 0
        self._free = list(range(self.pages - 1, used - 1, -1))
        return used
