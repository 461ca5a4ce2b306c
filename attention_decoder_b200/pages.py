"""Who holds which page of the K/V pool: leasing, sharing between forked slots, freeing and compaction.

The C ABI leaves the pool's pages to the caller; this is that caller's bookkeeping on the host (a reference count per
page). Device work goes through lfm3_reorder and lfm3_copy_pages."""
from __future__ import annotations

import numpy as np
import torch

from . import _lib as L

PAGE = 64


class Lfm3Pages:
    """Page pool of one ``Lfm3State``. Takes over the state's page table: every slot starts without pages.

    The full pages of a forked slot are shared with its source; the partly filled page that the next position goes to
    belongs to one slot alone. A call that writes positions below a slot's length (``restore``) needs pages of its own there:
    ``release`` and ``lease`` come first. All methods follow the host's view of the lengths (``state.h_seq_len``) and enqueue
    their device work on ``stream`` (default: torch's current stream)."""

    def __init__(self, state, stream=None):
        self.state, self.model = state, state.model
        self.refs = np.zeros(self.model.cfg.n_pages, dtype=np.int32)
        self.h = state.h_page_table
        self.h[:] = -1
        self._upload(stream)

    # ------------------------------------------------------------------ bookkeeping
    @property
    def free_pages(self) -> int:
        return int((self.refs == 0).sum())

    def _upload(self, stream=None, rows=slice(None)):
        with torch.cuda.stream(stream):
            self.state.page_table[rows].copy_(torch.from_numpy(self.h[rows]))

    def _take(self, n, candidates=None):
        """The n lowest free pages (or of the given candidates)."""
        free = np.flatnonzero(self.refs == 0 if candidates is None else candidates)
        if len(free) < n:
            raise L.Lfm3Error(-3, f"{n} pages are needed, {len(free)} of {len(self.refs)} are free")
        return free[:n].astype(np.int32)

    def _check(self, slot):
        if not 0 <= slot < self.h.shape[0]:  # (numpy counts negative ones from the end)
            raise L.Lfm3Error(-1, f"slot {slot} outside 0..{self.h.shape[0] - 1}")

    def lease(self, slot: int, positions: int, stream=None):
        """Makes sure that positions [0, positions) of ``slot`` have pages. Nothing changes on LFM3_E_CAPACITY."""
        self._check(slot)
        if positions < 0:
            raise L.Lfm3Error(-1, f"{positions} positions")
        need = (positions + PAGE - 1) // PAGE
        if need > self.h.shape[1]:
            raise L.Lfm3Error(-3, f"{positions} positions exceed the slot's {self.h.shape[1]} pages")
        missing = np.flatnonzero(self.h[slot, :need] < 0)
        if len(missing) == 0:
            return
        got = self._take(len(missing))
        self.h[slot, missing] = got
        self.refs[got] += 1
        self._upload(stream, slice(slot, slot + 1))

    def release(self, slot: int, stream=None):
        """Frees the slot for a new sequence: its pages lose one holder each, its length and conv columns become 0."""
        self._check(slot)
        row = self.h[slot]
        np.subtract.at(self.refs, row[row >= 0], 1)
        row[:] = -1
        self.state.h_seq_len[slot] = 0
        self._upload(stream, slice(slot, slot + 1))
        with torch.cuda.stream(stream):
            self.state.seq_len[slot: slot + 1].zero_()
            self.state.conv[:, slot].zero_()

    def reorder(self, slots, parents, stream=None):
        """lfm3_reorder with pages chosen here: slot slots[i] takes over the state of slot slots[parents[i]]."""
        slots, parents = [int(s) for s in slots], [int(p) for p in parents]
        if len(parents) != len(slots) or any(p < 0 or p >= len(slots) for p in parents):
            raise L.Lfm3Error(-1, "parents must be indices into slots, one for each slot")
        moved = [i for i, p in enumerate(parents) if p != i]
        if not moved:
            return
        length = self.state.h_seq_len
        refs = self.refs.copy()
        for i in moved:
            row = self.h[slots[i]]
            np.subtract.at(refs, row[row >= 0], 1)
        pages, fresh, given, sources = np.full(len(slots), -1, np.int32), [], set(), set()
        for i in moved:
            src = slots[parents[i]]
            full, part = int(length[src]) // PAGE, int(length[src]) % PAGE
            np.add.at(refs, self.h[src, :full], 1)
            if part:
                tail = int(self.h[src, full])
                if parents[parents[i]] != parents[i] and tail not in given:  # the parent's slot gives it up
                    pages[i] = tail
                    given.add(tail)
                    refs[tail] += 1
                else:
                    fresh.append(i)
                    sources.add(tail)
        free = refs == 0
        free[list(sources)] = False
        pages[fresh] = self._take(len(fresh), free)
        refs[pages[fresh]] += 1
        self.model.reorder(self.state, slots, parents, pages, stream=stream)
        self.refs = refs

    def fork(self, src: int, dsts, stream=None):
        """Slots ``dsts`` become copies of slot ``src`` that share its full pages."""
        dsts = list(dsts)
        self.reorder([src] + dsts, [0] * (1 + len(dsts)), stream=stream)

    def compact(self, stream=None) -> int:
        """Moves the pages in use to the lowest numbers, so that the pool's end is free; returns how many moved."""
        live = self.refs > 0
        n = int(live.sum())
        src = np.flatnonzero(live[n:]) + n
        if len(src) == 0:
            return 0
        dst = np.flatnonzero(~live[:n])
        self.model.copy_pages(self.state, src, dst, stream=stream)
        to = np.arange(len(self.refs), dtype=np.int32)
        to[src] = dst
        self.refs[dst], self.refs[src] = self.refs[src], 0
        self.h[:] = np.where(self.h >= 0, to[np.maximum(self.h, 0)], -1)
        self._upload(stream)
        return len(src)
