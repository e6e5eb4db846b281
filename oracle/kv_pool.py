"""Paged cache of the H2O oracle: sequences that share pages, in plain NumPy.

TEST INFRASTRUCTURE, like the rest of this package; it shares no code with the
CUDA path. One layer of a pool as the C header describes it: pages of keys,
values and positions, a page table, a length, a next position and accumulated
scores per sequence, and the number of holders of every page. The operators
change the arrays one list entry after the other, fp64 throughout; `errors`
collects the bits that the pool's error word would have.

The policy is that of the rest of the package: a compaction keeps, per head, the
r last tokens and the h others with the largest (score, position) keys, the
prompt selection of [H2O] appendix A (Pseudocode); accumulated scores are sums of
attention probabilities ([H2O] 1, 3.2).
"""
from __future__ import annotations

import numpy as np

from . import kv_fp8

BAD_STATE, BAD_LENGTH, NO_PAGE, BAD_LIST = 2, 4, 8, 16


def quantise(x):
    """kv_fp8.quantize_vector of every vector [..., d], those of magnitude up to 2^-119 as zero;
    one with a NaN or an infinity has zero codes and a NaN for its scale."""
    wild = ~np.isfinite(x).all(-1)
    x = np.where(wild[..., None], 0.0, x)
    amax = np.max(np.abs(x), -1).astype(np.float32)
    zero = amax <= 2.0 ** -119
    inv = np.float32(kv_fp8.E4M3_MAX) / np.where(zero, np.float32(1), amax)
    y = np.where(zero[..., None], np.float32(0), x.astype(np.float32) * inv[..., None])
    scale = np.where(zero, np.float32(0), amax / np.float32(kv_fp8.E4M3_MAX))
    return kv_fp8.e4m3_encode(y), np.where(wild, np.float32(np.nan), scale)


class Pool:
    """One layer. K, V hold the stored values (dequantised for fp8) in float64; with fp8 also
    the codes and scales."""

    def __init__(self, pages, page, heads, d, sequences, max_pages, fp8=False):
        self.page, self.heads, self.d, self.fp8 = page, heads, d, fp8
        self.width, self.cap = max_pages, max_pages * page
        shape = (pages, heads, page)
        self.K, self.V = np.zeros(shape + (d,)), np.zeros(shape + (d,))
        self.codes = {n: np.zeros(shape + (d,), np.uint8) for n in "KV"}
        self.scale = {n: np.zeros(shape, np.float32) for n in "KV"}
        self.pos = np.full(shape, -1, np.int32)
        self.score = np.zeros((sequences, heads, self.cap))
        self.table = np.full((sequences, max_pages), -1, np.int32)
        self.meta = np.zeros((sequences, 2), np.int32)
        self.ref = np.zeros(pages, np.int32)
        self.errors = 0

    # ------------------------------------------------------------------ pages
    def _need(self, tokens):
        return -(-tokens // self.page)

    def _take(self, n):
        free = np.flatnonzero(self.ref == 0)[:n]
        assert len(free) == n
        self.ref[free] = 1
        return free

    def _serve(self, needs):
        """How many list entries the free pages serve, in order."""
        free = int(np.sum(self.ref == 0))
        for i, n in enumerate(needs):
            free -= n
            if free < 0:
                self.errors |= NO_PAGE
                return i
        return len(needs)

    def _list(self, seqs):
        """The list with the entries that cannot be meant replaced by -1."""
        seen, out = set(), []
        for s in seqs:
            s = int(s)
            bad = s != -1 and (s < 0 or s >= len(self.meta) or s in seen)
            if bad:
                self.errors |= BAD_LIST
            seen.add(s)
            out.append(-1 if bad else s)
        return out

    def _slots(self, seq, n=None):
        """(pages, offsets) of a sequence's first n tokens."""
        j = np.arange(int(self.meta[seq, 0]) if n is None else n)
        return self.table[seq][j // self.page], j % self.page

    def _move(self, to, to_off, at, at_off, head=slice(None)):
        for x in (self.K, self.V, self.pos, self.codes["K"], self.codes["V"], self.scale["K"],
                  self.scale["V"]):
            x[to, head, to_off] = x[at, head, at_off]

    # -------------------------------------------------------------- operators
    def write(self, seqs, K, V, lens=None, score=None):
        """K, V float64 [n, heads, T, d]."""
        T = K.shape[2]
        seqs = self._list(seqs)
        todo = []
        for i, s in enumerate(seqs):
            if s < 0:
                continue
            t = T if lens is None else int(lens[i])
            if not 0 <= t <= T:
                self.errors |= BAD_LENGTH
                t = min(max(t, 0), T)
            if self.meta[s, 0] + t > self.cap:
                self.errors |= NO_PAGE
                continue
            todo.append((i, s, t, self._need(self.meta[s, 0] + t) - self._need(self.meta[s, 0])))
        for i, s, t, need in todo[:self._serve([x[3] for x in todo])]:
            have, first = (int(x) for x in self.meta[s])
            self.table[s, self._need(have):self._need(have) + need] = self._take(need)
            self.meta[s] += t
            j = np.arange(t)
            p, o = self.table[s][(have + j) // self.page], (have + j) % self.page
            for name, store, new in (("K", self.K, K), ("V", self.V, V)):
                x = new[i, :, :t].swapaxes(0, 1)  # [t, heads, d]
                if self.fp8:
                    c, sc = quantise(x)
                    self.codes[name][p, :, o], self.scale[name][p, :, o] = c, sc
                    x = kv_fp8.dequantize_vector(c, sc[..., None])
                store[p, :, o] = x
            self.pos[p, :, o] = (first + j)[:, None]
            self.score[s, :, have:have + t] = 0 if score is None else score[i, :, :t]

    def fork(self, src, dst, share=True):
        dst = self._list(dst)
        meta, todo = self.meta.copy(), []
        for a, b in zip(src, dst):
            a = int(a)
            if b < 0 or a == -1:
                continue
            if not 0 <= a < len(meta) or meta[b, 0] != 0:
                self.errors |= BAD_LIST
                continue
            n = int(meta[a, 0])
            todo.append((a, b, n, int(n % self.page > 0) if share else self._need(n)))
        for a, b, n, need in todo[:self._serve([x[3] for x in todo])]:
            whole = n // self.page if share else 0
            self.ref[self.table[a, :whole]] += 1
            self.table[b, :whole] = self.table[a, :whole]
            self.table[b, whole:whole + need] = self._take(need)
            for j in range(whole * self.page, n):
                self._move(self.table[b, j // self.page], j % self.page,
                           self.table[a, j // self.page], j % self.page)
            self.meta[b] = meta[a]
            self.score[b, :, :n] = self.score[a, :, :n]

    def free(self, seqs):
        for s in self._list(seqs):
            if s < 0:
                continue
            held = self.table[s, :self._need(self.meta[s, 0])]
            self.ref[held] -= 1
            self.table[s], self.meta[s] = -1, 0

    def compact(self, seqs, h, r):
        k = h + r
        todo = [(s, self._need(k)) for s in self._list(seqs) if s >= 0 and self.meta[s, 0] > k]
        todo = todo[:self._serve([x[1] for x in todo])]
        fresh = [self._take(need) for _, need in todo]
        for (s, _), new in zip(todo, fresh):
            n = int(self.meta[s, 0])
            pages, offs = self._slots(s)
            for head in range(self.heads):
                old = self.score[s, head, :n]
                order = sorted(range(n - r), key=lambda j: (np.isnan(old[j]), np.nan_to_num(old[j]), j))
                kept = np.array(sorted(order[n - r - h:]) + list(range(n - r, n)), dtype=np.int64)
                j = np.arange(k)
                self._move(new[j // self.page], j % self.page, pages[kept], offs[kept], head)
                self.score[s, head, :k] = old[kept].copy()
            self.ref[self.table[s, :self._need(n)]] -= 1
            self.table[s] = -1
            self.table[s, :len(new)] = new
            self.meta[s, 0] = k

    def attend(self, seqs, q, prefix=-1, accumulate=True):
        """q float64 [n, q_heads, d]; (out, lse) with NaN in rows that are not written."""
        group = q.shape[1] // self.heads
        out, lse = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
        P = int(self.meta[prefix, 0]) if prefix >= 0 else 0
        shared = self._slots(prefix) if prefix >= 0 else None
        added = np.zeros((self.heads, P))
        for i, s in enumerate(self._list(seqs)):
            if s < 0:
                continue
            if s == prefix:
                self.errors |= BAD_LIST
                continue
            n = int(self.meta[s, 0])
            pages, offs = self._slots(s)
            if shared is not None:
                pages, offs = np.concatenate([shared[0], pages]), np.concatenate([shared[1], offs])
            for hq in range(q.shape[1]):
                h = hq // group
                if not len(pages):
                    out[i, hq], lse[i, hq] = 0, -np.inf
                    continue
                x = self.K[pages, h, offs] @ q[i, hq] / np.sqrt(self.d)
                top = x.max()
                e = np.exp(x - top)
                p = e / e.sum()
                out[i, hq], lse[i, hq] = p @ self.V[pages, h, offs], top + np.log(e.sum())
                if accumulate:
                    added[h] += p[:P]
                    self.score[s, h, :n] += p[P:]
        if accumulate and prefix >= 0:
            self.score[prefix, :, :P] += added
        return out, lse
