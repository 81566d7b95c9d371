"""Sequences over a paged 8-bit K/V cache (KV8): which pages each one owns,
and the appends, forks, truncations and moves that keep it so.

Host logic only; the codes are written by lsa_kv8_write and moved by
lsa_kv8_copy_pages.  A page belongs to every sequence whose table names it
(a reference count); a fork shares the pages of its parent's tokens, and the first
append of either into a shared page that is still open copies it first.  Pages
that `reserve` promised to a writer are never shared: a fork gets its own copy of
an open page that tokens are still to be written into.
Free pages are handed out lowest number first, so that `compact` has little
to move.  The calls are taken from an `ops` object, as in `seqshard`, so that
the tests run the same logic without a GPU.

Nothing changes when a call is refused: the pages and copies of an append are
planned first, then the device calls are made, then the sequences change.  Device
work is ordered by the stream of each call: use one stream, or order them.
"""
from __future__ import annotations

import heapq
import itertools

import torch

from ._lib import LSA_ENOSPACE, LSAError


class LibraryOps:
    """The library's calls (CUDA tensors)."""

    def write(self, kv, K, V, table, start, cu, stream):
        from . import api
        api.kv8_write(kv, K, V, table, start, cu=cu, stream=stream)

    def copy(self, kv, src, dst, stream):
        from . import api
        api.kv8_copy_pages(kv, src, dst, stream=stream)


class _Sequence:
    __slots__ = ("pages", "len", "reserved")  # reserved: tokens that `advance` may still count

    def __init__(self, pages, n):
        self.pages, self.len, self.reserved = pages, n, 0


class KV8Pages:
    """The sequences of one cache.  `kv`: a KV8."""

    def __init__(self, kv, ops=None):
        self.kv = kv
        self.ops = ops or LibraryOps()
        self.refs = [0] * kv.n_pages
        self._free = list(range(kv.n_pages))  # a heap: lowest number first
        self._seqs: dict[int, _Sequence] = {}
        self._next = 0

    # ------------------------------------------------------------ state

    @property
    def free_pages(self) -> int:
        return len(self._free)

    @property
    def used_pages(self) -> int:
        return self.kv.n_pages - len(self._free)

    def _seq(self, sid) -> _Sequence:
        if sid not in self._seqs:
            raise ValueError(f"no sequence {sid}")
        return self._seqs[sid]

    def __contains__(self, sid) -> bool:
        return sid in self._seqs

    def len(self, sid) -> int:
        """Tokens of a sequence."""
        return self._seq(sid).len

    def pages(self, sid) -> list[int]:
        """Its pages, in order."""
        return list(self._seq(sid).pages)

    def _upload(self, rows):
        t = torch.tensor(rows, dtype=torch.int32)
        if self.kv.device.type == "cuda":
            t = t.pin_memory().to(self.kv.device, non_blocking=True)
        return t

    def table(self, sids, width: int | None = None):
        """(table [n, width], lens [n]) of these sequences, int32 on the cache's
        device, for the attention calls.  width: at least the longest's pages
        (the default)."""
        seqs = [self._seq(s) for s in sids]
        need = max([len(s.pages) for s in seqs], default=0)
        width = max(1, need) if width is None else width
        if width < need:
            raise ValueError(f"width: a sequence holds {need} pages, got {width}")
        return (self._upload([s.pages + [-1] * (width - len(s.pages)) for s in seqs]).view(len(seqs), width),
                self._upload([s.len for s in seqs]))

    # ------------------------------------------------------ life of a page

    def _release(self, pages):
        for p in pages:
            self.refs[p] -= 1
            if self.refs[p] == 0:
                heapq.heappush(self._free, p)

    def add(self) -> int:
        """A new, empty sequence."""
        sid, self._next = self._next, self._next + 1
        self._seqs[sid] = _Sequence([], 0)
        return sid

    def fork(self, sid, stream=None) -> int:
        """A sequence with the same tokens, sharing their pages.  What the parent
        reserved stays its own: if tokens are still to be written into its open
        page, the fork gets a copy of that page (LSA_ENOSPACE without a free one)."""
        parent = self._seq(sid)
        pages = parent.pages[:-(-parent.len // self.kv.page)]
        if parent.reserved and parent.len % self.kv.page:
            if not self._free:
                raise LSAError(LSA_ENOSPACE, f"fork: sequence {sid} holds reserved tokens and no page is free for its open page's copy")
            own = heapq.heappop(self._free)
            try:
                self.ops.copy(self.kv, [pages[-1]], [own], stream)
            except BaseException:
                heapq.heappush(self._free, own)
                raise
            pages[-1] = own
        for p in pages:
            self.refs[p] += 1
        new = self.add()
        self._seqs[new] = _Sequence(pages, parent.len)
        return new

    def free(self, sid):
        """Forget a sequence; pages nobody else names become free."""
        self._release(self._seq(sid).pages)
        del self._seqs[sid]

    def truncate(self, sid, n: int):
        """Keep a sequence's first n tokens (rejected drafts) and nothing that
        is reserved.  An open page keeps its scale."""
        seq = self._seq(sid)
        if not 0 <= n <= seq.len:
            raise ValueError(f"truncate: sequence {sid} holds {seq.len} tokens, got {n}")
        keep = -(-n // self.kv.page)
        self._release(seq.pages[keep:])
        seq.pages, seq.len, seq.reserved = seq.pages[:keep], n, 0

    def _counts(self, what, sids, counts):
        sids = list(sids)
        seqs = [self._seq(s) for s in sids]
        if len(set(sids)) < len(sids):
            raise ValueError(f"{what}: a sequence stands twice")
        counts = [1] * len(sids) if counts is None else [int(c) for c in counts]
        if len(counts) != len(sids) or any(c < 0 for c in counts):
            raise ValueError(f"{what}: counts must be one non-negative number a sequence")
        return seqs, counts

    def _own(self, what, seqs, counts, stream, then=None):
        """Give every sequence pages of its own for its next tokens: a copy of
        a shared open page, new pages behind it; then run `then(tables)`.  What
        the sequences hold changes only when all of it has been done."""
        page = self.kv.page
        given: dict[int, int] = {}      # references to shared pages that are given up
        copies: list[tuple[int, int]] = []
        tables, taken, short = [], [], 0
        for seq, c in zip(seqs, counts):
            pages = list(seq.pages)
            want = [None] * max(0, -(-(seq.len + c) // page) - len(pages))
            if c > 0 and seq.len % page:
                at = seq.len // page
                p = pages[at]
                if self.refs[p] - given.get(p, 0) > 1:
                    given[p] = given.get(p, 0) + 1
                    pages[at] = None
            pages += want
            for i, p in enumerate(pages):
                if p is not None:
                    continue
                if self._free:
                    pages[i] = heapq.heappop(self._free)
                    taken.append(pages[i])
                    if i < len(seq.pages):
                        copies.append((seq.pages[i], pages[i]))
                else:
                    short += 1
            tables.append(pages)
        try:
            if short:
                raise LSAError(LSA_ENOSPACE, f"{what}: {short} more free pages are needed than the {len(taken)} there are")
            if copies:
                self.ops.copy(self.kv, [s for s, _ in copies], [d for _, d in copies], stream)
            if then is not None:
                then(tables)
        except BaseException:
            for p in taken:
                heapq.heappush(self._free, p)
            raise
        for p in taken:
            self.refs[p] = 1
        for p, n in given.items():
            self.refs[p] -= n
        for seq, pages in zip(seqs, tables):
            seq.pages = pages

    @staticmethod
    def _count(seqs, counts):
        for seq, c in zip(seqs, counts):
            seq.len += c
            seq.reserved = max(0, seq.reserved - c)

    def append(self, sids, K, V, counts=None, stream=None):
        """Write new tokens: K, V [n, hkv, 128] bf16, counts[i] rows for
        sequence sids[i] (default one each), in order.  LSA_ENOSPACE if the free
        pages do not suffice."""
        seqs, counts = self._counts("append", sids, counts)
        shape = (sum(counts), self.kv.hkv, 128)
        for name, t in (("K", K), ("V", V)):
            if tuple(t.shape) != shape:
                raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
            if t.dtype != torch.bfloat16:
                raise TypeError(f"{name}: expected {torch.bfloat16}, got {t.dtype}")

        def write(tables):
            width = max(len(p) for p in tables)
            up = stream if self.kv.device.type == "cuda" else None
            with torch.cuda.stream(up):  # the tables are uploaded where they are read
                table = self._upload([p + [-1] * (width - len(p)) for p in tables]).view(len(tables), width)
                start = self._upload([s.len for s in seqs])
                cu = None
                if any(c != 1 for c in counts):
                    cu = self._upload([0, *itertools.accumulate(counts)])
                self.ops.write(self.kv, K, V, table, start, cu, stream)

        self._own("append", seqs, counts, stream, write if shape[0] else None)
        self._count(seqs, counts)

    def reserve(self, sids, counts=None, stream=None):
        """Pages for the next counts[i] tokens of sequence sids[i] (default one
        each) that something else writes, a decode step for one: `table` names
        them afterwards.  Tell with `advance` how many were written."""
        seqs, counts = self._counts("reserve", sids, counts)
        self._own("reserve", seqs, counts, stream)
        for seq, c in zip(seqs, counts):
            seq.reserved = max(seq.reserved, c)

    def advance(self, sids, counts=None):
        """Count tokens that were written into reserved pages.  Refused where
        one of these pages belongs to another sequence too."""
        sids = list(sids)
        seqs, counts = self._counts("advance", sids, counts)
        for sid, seq, c in zip(sids, seqs, counts):
            if seq.len + c > len(seq.pages) * self.kv.page:
                raise ValueError(f"advance: sequence {sid} has pages for {len(seq.pages) * self.kv.page} tokens, not {seq.len + c}")
            if c > 0 and any(self.refs[p] > 1 for p in seq.pages[seq.len // self.kv.page:-(-(seq.len + c) // self.kv.page)]):
                raise ValueError(f"advance: sequence {sid} shares a page that the tokens would stand in (reserve them first)")
        self._count(seqs, counts)

    def compact(self, stream=None) -> int:
        """Move the used pages to the lowest numbers.  Returns how many moved;
        afterwards the pages from used_pages on are free.  Tables made before
        are void."""
        used = self.used_pages
        src = [p for p in range(used, self.kv.n_pages) if self.refs[p] > 0]
        dst = sorted(p for p in self._free if p < used)
        if not src:
            return 0
        self.ops.copy(self.kv, src, dst, stream)
        to = dict(zip(src, dst))
        for seq in self._seqs.values():
            seq.pages = [to.get(p, p) for p in seq.pages]
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        self._free = list(range(used, self.kv.n_pages))
        return len(src)
