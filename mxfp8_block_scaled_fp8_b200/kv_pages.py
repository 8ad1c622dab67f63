"""Bookkeeping of a key/value cache's pages on the host: which are free, which
are shared by several sequences, and which page copies a fork or a compaction
needs.  It holds page numbers only; ``kv_copy_pages`` moves the bytes (in all
layers at once), and the caller keeps each sequence's list of pages, the rows
of its page table.

    pool = KvPagePool(cache.shape[-2], page_size)
    pages = pool.allocate(pool.pages_for(length))
    child, src, dst = pool.fork(pages, length)       # shares full pages
    fp8mm.kv_copy_pages(cache, src, dst)
    src, dst, moved = pool.compact()                 # live pages to the front
    fp8mm.kv_copy_pages(cache, src, dst)
    pages = [moved.get(p, p) for p in pages]         # every list of pages
"""
from __future__ import annotations

import heapq


class KvPagePool:
    def __init__(self, num_pages: int, page_size: int):
        if num_pages < 0 or page_size < 16 or page_size % 16 != 0 or page_size > 4096:
            raise ValueError(f"{num_pages} pages of {page_size} tokens")
        self.num_pages, self.page_size = num_pages, page_size
        self._refs = [0] * num_pages
        self._free = list(range(num_pages))  # a heap: the lowest page is taken first

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def pages_for(self, length: int) -> int:
        """Pages that a sequence of this length takes."""
        if length < 0:
            raise ValueError(f"length {length}")
        return -(-length // self.page_size)

    def references(self, page: int) -> int:
        """Sequences that hold the page."""
        return self._refs[self._page(page)]

    def allocate(self, n: int) -> list[int]:
        """n free pages, each with one holder; MemoryError, and nothing taken, if there are fewer."""
        if n < 0:
            raise ValueError(f"{n} pages")
        if n > len(self._free):
            raise MemoryError(f"{n} pages asked for, {len(self._free)} free")
        pages = [heapq.heappop(self._free) for _ in range(n)]
        for p in pages:
            self._refs[p] = 1
        return pages

    def free(self, pages) -> None:
        """One holder gives these pages up (a sequence ends); a page without holders is free again.  ValueError, and
        nothing given up, for a page that has fewer holders."""
        pages = list(pages)
        less: dict[int, int] = {}
        for p in pages:
            less[self._page(p)] = less.get(p, 0) + 1
        for p, n in less.items():
            if n > self._refs[p]:
                raise ValueError(f"page {p} has {self._refs[p]} holders, {n} give it up")
        for p, n in less.items():
            self._refs[p] -= n
            if self._refs[p] == 0:
                heapq.heappush(self._free, p)

    def fork(self, pages, length: int):
        """A second holder of a sequence of this length: (its pages, src, dst).  Full pages are shared, since tokens are
        only appended; a partly filled last page is copied, and kv_copy_pages(cache, src, dst) has to run before either
        sequence appends.  Pages behind the length are not taken over."""
        pages = list(pages)
        n = self.pages_for(length)
        if n > len(pages):
            raise ValueError(f"{len(pages)} pages do not hold {length} tokens")
        for p in pages[:n]:
            if self._refs[self._page(p)] == 0:
                raise ValueError(f"page {p} is free")
        full = length // self.page_size
        child, src, dst = pages[:full], [], []
        if full < n:
            dst = self.allocate(1)
            src = [pages[full]]
            child.append(dst[0])
        for p in pages[:full]:
            self._refs[p] += 1
        return child, src, dst

    def compact(self):
        """Moves the held pages to the lowest numbers: (src, dst, {old page: new page}) of the pages that move.  The
        copies are independent of one another: every dst was free."""
        held = self.num_pages - len(self._free)
        dst = sorted(p for p in self._free if p < held)
        src = [p for p in range(held, self.num_pages) if self._refs[p] > 0]
        for old, new in zip(src, dst, strict=True):
            self._refs[new], self._refs[old] = self._refs[old], 0
        self._free = list(range(held, self.num_pages))
        return src, dst, dict(zip(src, dst))

    def _page(self, p: int) -> int:
        if not 0 <= p < self.num_pages:
            raise ValueError(f"page {p} of {self.num_pages}")
        return p
