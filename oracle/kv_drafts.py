"""Drafted tokens over the paged cache of the H2O oracle, in plain NumPy and fp64.

TEST INFRASTRUCTURE, like the rest of this package. The operators of kv_pool.Pool, and: tokens
appended with their positions' rotation, attention of a tree of drafts, and what is kept of them.
"""
from __future__ import annotations

import numpy as np

from . import kv_fp8, rotary
from .kv_pool import BAD_LENGTH, BAD_LIST, BAD_STATE, NO_PAGE, Pool, quantise


class DraftPool(Pool):
    """refused: by sequence, REFUSED where its last write or append was not served, QUERIES too where
    that was an append with queries."""

    REFUSED, QUERIES = 1, 2

    def __init__(self, pages, page, heads, d, sequences, max_pages, fp8=False):
        super().__init__(pages, page, heads, d, sequences, max_pages, fp8)
        self.refused = np.zeros(sequences, np.int32)

    def _mark(self, seqs, T, lens, before, mark):
        """Entries whose tokens did not come have `mark`, the others none."""
        errors = self.errors
        for i, s in enumerate(self._list(seqs)):
            if s >= 0:
                t = self._lens(T, lens, i)
                self.refused[s] = mark if t > 0 and self.meta[s, 0] == before[s] else 0
        self.errors = errors

    def write(self, seqs, K, V, lens=None, score=None):
        before = self.meta[:, 0].copy()
        super().write(seqs, K, V, lens, score)
        self._mark(seqs, K.shape[2], lens, before, self.REFUSED)

    def fork(self, src, dst, share=True):
        before, free, errors = self.meta[:, 0].copy(), int(np.sum(self.ref == 0)), self.errors
        for a, b in zip(src, self._list(dst)):
            if b >= 0 and 0 <= a < len(before) and before[b] == 0:
                free -= int(before[a] % self.page > 0) if share else self._need(before[a])
                if free < 0:
                    break
                self.refused[b] = 0
        self.errors = errors
        super().fork(src, dst, share)

    def free(self, seqs):
        super().free(seqs)
        self.refused[[s for s in seqs if 0 <= s < len(self.refused)]] = 0

    def attend(self, seqs, q, prefix=-1, accumulate=True):
        seqs = [-1 if s >= 0 and s != prefix and self.refused[s] & self.QUERIES else s for s in self._list(seqs)]
        return super().attend(seqs, q, prefix, accumulate)

    def _lens(self, T, lens, i):
        t = T if lens is None else int(lens[i])
        if not 0 <= t <= T:
            self.errors |= BAD_LENGTH
            t = min(max(t, 0), T)
        return t

    def append(self, seqs, T, lens, parent, make, queries=True):
        """make(i, positions) gives keys and values float64 [heads, tokens, d] of entry i before they are
        stored. Returns {entry: positions}."""
        todo, got, before = [], {}, self.meta[:, 0].copy()
        for i, s in enumerate(self._list(seqs)):
            if s < 0:
                continue
            t = self._lens(T, lens, i)
            if self.meta[s, 0] + t > self.cap:
                self.errors |= NO_PAGE
                continue
            todo.append((i, s, t, self._need(self.meta[s, 0] + t) - self._need(self.meta[s, 0])))
        for i, s, t, need in todo[:self._serve([x[3] for x in todo])]:
            have, first = (int(x) for x in self.meta[s])
            self.table[s, self._need(have):self._need(have) + need] = self._take(need)
            ahead = np.arange(t)
            if parent is not None:
                up = [int(x) for x in parent[i][:t]]
                if any(not -1 <= p < j for j, p in enumerate(up)):
                    self.errors |= BAD_LIST
                ahead = np.array(rotary.depths(up), dtype=np.int64)
            got[i] = first + ahead
            K, V = make(i, got[i])
            p, o = self._at(s, have + np.arange(t))
            for name, store, x in (("K", self.K, K), ("V", self.V, V)):
                x = x.swapaxes(0, 1)
                if self.fp8:
                    c, sc = quantise(x)
                    self.codes[name][p, :, o], self.scale[name][p, :, o] = c, sc
                    x = kv_fp8.dequantize_vector(c, sc[..., None])
                store[p, :, o] = x
            self.pos[p, :, o] = got[i][:, None]
            self.score[s, :, have:have + t] = 0
            self.meta[s] += (t, 0 if parent is not None else t)
        self._mark(seqs, T, lens, before, self.REFUSED | (self.QUERIES if queries else 0))
        return got

    def _at(self, seq, slots):
        slots = np.asarray(slots, dtype=np.int64)
        return self.table[seq][slots // self.page], slots % self.page

    def _keys(self, seq, slots, head):
        p, o = self._at(seq, slots)
        return self.K[p, head, o], self.V[p, head, o]

    def attend_tree(self, seqs, q, prefix=-1, lens=None, parent=None):
        """q float64 [n, T, q_heads, d]; (out, lse) with NaN in rows that are not written."""
        n, T, q_heads, d = q.shape
        group = q_heads // self.heads
        out, lse = np.full(q.shape, np.nan), np.full(q.shape[:3], np.nan)
        P = int(self.meta[prefix, 0]) if prefix >= 0 else 0
        for i, s in enumerate(self._list(seqs)):
            if s < 0:
                continue
            if s == prefix:
                self.errors |= BAD_LIST
                continue
            if self.refused[s]:
                continue
            nodes, length = self._lens(T, lens, i), int(self.meta[s, 0])
            if nodes > length:
                self.errors |= BAD_LENGTH
                continue
            up = list(range(-1, nodes - 1)) if parent is None else [int(x) for x in parent[i][:nodes]]
            if any(not -1 <= p < j for j, p in enumerate(up)):
                self.errors |= BAD_LIST
            base = length - nodes
            for t in range(nodes):
                slots = list(range(base)) + [base + j for j in rotary.branch(up, t)]
                for hq in range(q_heads):
                    k, v = self._keys(s, slots, hq // group)
                    if P:
                        pk, pv = self._keys(prefix, range(P), hq // group)
                        k, v = np.concatenate([pk, k]), np.concatenate([pv, v])
                    x = k @ q[i, t, hq] / np.sqrt(d)
                    top = x.max()
                    e = np.exp(x - top)
                    out[i, t, hq], lse[i, t, hq] = e / e.sum() @ v, top + np.log(e.sum())
        return out, lse

    def accept(self, seqs, T, path=None, lens=None, q=None, lse=None, prefix=-1):
        """q float64 [n, T, q_heads, d] and lse [n, T, q_heads]: what the scores grow by."""
        added = None
        for i, s in enumerate(self._list(seqs)):
            if s < 0:
                continue
            if s == prefix and q is not None:
                self.errors |= BAD_LIST
                continue
            if self.refused[s]:
                self.refused[s] = 0
                continue
            nodes, length = self._lens(T, lens, i), int(self.meta[s, 0])
            if nodes > length:
                self.errors |= BAD_LENGTH
                continue
            kept = [] if path is None else [int(x) for x in path[i]]
            count = next((j for j, x in enumerate(kept) if x < 0), len(kept))
            kept, rest = kept[:count], kept[count:]
            if any(x != -1 for x in rest) or any(b <= a for a, b in zip([-1] + kept, kept)) or (kept and kept[-1] >= nodes):
                self.errors |= BAD_LIST
                continue
            base = length - nodes
            if nodes == 0:
                continue
            written = self.table[s, base // self.page:self._need(base + count)]
            if np.any(self.ref[written] != 1):
                self.errors |= BAD_STATE
                continue
            p, o = self._at(s, [base])
            first = int(self.pos[p[0], 0, o[0]])
            if kept:
                old, new = self._at(s, [base + x for x in kept]), self._at(s, base + np.arange(count))
                self._move(new[0], new[1], old[0].copy(), old[1].copy())
            keep = self._need(base + count)
            gone = self.table[s, keep:self._need(length)].copy()
            self.ref[gone] -= 1
            self.table[s, keep:] = -1
            self.meta[s] = (base + count, first + count)
            self.score[s, :, base:base + count] = 0
            if q is None:
                continue
            group = q.shape[2] // self.heads
            P = int(self.meta[prefix, 0]) if prefix >= 0 else 0
            if added is None:
                added = np.zeros((self.heads, P))
            for j, x in enumerate(kept):
                for hq in range(q.shape[2]):
                    if lse[i, x, hq] == -np.inf:
                        continue
                    h, scale = hq // group, np.sqrt(self.d)
                    k, _ = self._keys(s, range(base + j + 1), h)
                    self.score[s, h, :base + j + 1] += np.exp(k @ q[i, x, hq] / scale - lse[i, x, hq])
                    if P:
                        k, _ = self._keys(prefix, range(P), h)
                        added[h] += np.exp(k @ q[i, x, hq] / scale - lse[i, x, hq])
        if added is not None and prefix >= 0:
            self.score[prefix, :, :added.shape[1]] += added
