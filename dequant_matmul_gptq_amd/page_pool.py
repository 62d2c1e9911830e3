"""Host bookkeeping of a paged cache's pages: who holds which page, and which
copies the caches need. Sequences share pages by reference counts; the layers
of a model share one page numbering, so one pool serves all of their caches.
Nothing here touches a GPU: the calls return (source, target) pairs for
copy_pages, to be run before the sequences are appended to.
"""

from __future__ import annotations


class PagePool:
    """Pages 0 .. num_pages - 1 of page_size token slots each.

    A sequence is a key the caller picks; its page list is `pages(seq)` and its
    token count `length(seq)`. A page held by several sequences is full and
    never appended to: fork gives the copy its own last page if that one is
    only partly filled, or cut.
    """

    def __init__(self, num_pages: int, page_size: int):
        if num_pages < 1 or page_size < 1:
            raise ValueError("a pool needs at least one page of at least one slot")
        self.num_pages, self.page_size = int(num_pages), int(page_size)
        self._free = list(range(self.num_pages - 1, -1, -1))    # popped from the end: lowest page first
        self._refs = [0] * self.num_pages
        self._pages: dict = {}
        self._length: dict = {}

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def sequences(self) -> list:
        return list(self._pages)

    def pages(self, seq) -> list[int]:
        return list(self._pages[seq])

    def length(self, seq) -> int:
        return self._length[seq]

    def _take(self) -> int:
        p = self._free.pop()
        self._refs[p] = 1
        return p

    def _drop(self, p: int) -> None:
        self._refs[p] -= 1
        if self._refs[p] == 0:
            self._free.append(p)

    def add(self, seq) -> None:
        """A new, empty sequence."""
        if seq in self._pages:
            raise ValueError(f"sequence {seq!r} is already in the pool")
        self._pages[seq], self._length[seq] = [], 0

    def extend(self, seq, tokens: int) -> list[int]:
        """Room for `tokens` more tokens: their slots, in order. Raises
        MemoryError, changing nothing, if the pool has too few free pages."""
        if tokens < 0:
            raise ValueError("tokens must not be negative")
        pages, at, P = self._pages[seq], self._length[seq], self.page_size
        need = -(-(at + tokens) // P) - len(pages)
        if need > len(self._free):
            raise MemoryError(f"{need} pages needed, {len(self._free)} free")
        for _ in range(need):
            pages.append(self._take())
        self._length[seq] = at + tokens
        return [pages[t // P] * P + t % P for t in range(at, at + tokens)]

    def truncate(self, seq, length: int) -> None:
        """Forget the tokens from `length` on (rejected drafts). A shared page
        that would become partly filled cannot be appended to, so that is
        refused: fork the sequence up to `length` and free it instead."""
        if not 0 <= length <= self._length[seq]:
            raise ValueError("length must be between 0 and the sequence's own")
        pages, P = self._pages[seq], self.page_size
        keep = -(-length // P)
        if length % P and self._refs[pages[keep - 1]] > 1:
            raise ValueError("the sequence would end inside a shared page: fork it up to that length")
        for p in pages[keep:]:
            self._drop(p)
        del pages[keep:]
        self._length[seq] = length

    def fork(self, seq, new, length: int | None = None) -> list[tuple[int, int]]:
        """`new` starts as a copy of the first `length` tokens of `seq` (None:
        all): full pages are shared, a page that they fill in part is copied.
        Returns the copies to run (none or one)."""
        if new in self._pages:
            raise ValueError(f"sequence {new!r} is already in the pool")
        length = self._length[seq] if length is None else length
        if not 0 <= length <= self._length[seq]:
            raise ValueError("length must be between 0 and the sequence's own")
        full, part = divmod(length, self.page_size)
        pages = self._pages[seq][:full]
        copies = []
        if part:
            if not self._free:
                raise MemoryError("1 page needed, 0 free")
            copies.append((self._pages[seq][full], self._take()))
        for p in pages:
            self._refs[p] += 1
        self._pages[new], self._length[new] = pages + [p for _, p in copies], length
        return copies

    def free(self, seq) -> None:
        """Drop a sequence; pages that nobody else holds become free."""
        for p in self._pages.pop(seq):
            self._drop(p)
        del self._length[seq]

    def compact(self) -> list[tuple[int, int]]:
        """Move the pages in use to the lowest numbers. Returns the copies to
        run: every target is a free page and every source lies above them all,
        so no page appears twice."""
        used = self.num_pages - len(self._free)
        targets = [p for p in range(used) if self._refs[p] == 0]
        sources = [p for p in range(used, self.num_pages) if self._refs[p] > 0]
        moved = dict(zip(sources, targets))
        for s, t in moved.items():
            self._refs[t], self._refs[s] = self._refs[s], 0
        for pages in self._pages.values():
            pages[:] = [moved.get(p, p) for p in pages]
        self._free = list(range(self.num_pages - 1, used - 1, -1))
        return list(moved.items())
