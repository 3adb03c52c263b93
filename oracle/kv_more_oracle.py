"""Capped and biased attention with document and prefix masks, compaction and the page pool, from the definitions (numpy and
plain Python, no GPU code shared). Caches and rows are as in kv_oracle."""
from __future__ import annotations

import numpy as np

from .kv_oracle import least_scale, to_e4m3, visible


def sees(p: int, n: int, window=0, sinks=0, doc_start=None, prefix_end=None, listed=None, entry_tokens=1) -> np.ndarray:
    """Which of the n cached positions the query at p sees."""
    s = np.arange(n)
    upto = p if prefix_end is None else max(p, prefix_end - 1)
    if listed is None and window == 0:
        see = s <= upto
    else:
        see = visible(p, n, window, sinks, listed, entry_tokens)  # a prefix has no window
    return see if doc_start is None else see & (s >= doc_start)


def scores(y: np.ndarray, p: int, softcap=0.0, slope=0.0) -> np.ndarray:
    """The scores of positions 0 .. n - 1 from y = scale q . K_s."""
    with np.errstate(invalid="ignore", over="ignore"):
        x = softcap * np.tanh(y / softcap) if softcap else np.array(y)
    return x - slope * np.abs(p - np.arange(len(x)))


def attend_row(q, K, V, see, p, scale, softcap=0.0, slope=0.0):
    """One query row: (out [d], lse, sum_s P_s |V_s| [d], largest sum |q_i K_si| |scale|, largest |bias| of a seen key)."""
    d = V.shape[1]
    if not see.any():
        return np.zeros(d), -np.inf, np.zeros(d), 0.0, 0.0
    with np.errstate(invalid="ignore", over="ignore"):
        x = scores(K @ q * scale, p, softcap, slope)[see]
        v = V[see]
        m = x.max()
        w = np.exp(x - m)
        l = w.sum()
        far = np.abs(p - np.flatnonzero(see)).max()
        big = (np.abs(K[see]) @ np.abs(q)).max() * abs(scale)
        return w @ v / l, m + np.log(l), w @ np.abs(v) / l, float(big), float(abs(slope) * far)


def kept_positions(length: int, listed, entry_tokens: int, window: int, sinks: int) -> list:
    listed = set(int(e) for e in listed)
    return [s for s in range(length) if s // entry_tokens in listed or s < sinks or s >= length - window]


def compact_page(values: np.ndarray):
    """e4m3 codes and scale of one new page and head; values [n, d] with NaN where the old code was NaN."""
    fin = values[np.isfinite(values)]
    scale = least_scale(np.abs(fin).max(initial=0.0))
    return to_e4m3(values / scale), scale


class Pool:
    """refs, table and kv_len as lists; every call does what the library's does, one page at a time."""

    def __init__(self, refs, table, kv_len, page_tokens):
        self.refs, self.table, self.kv_len, self.pt = list(refs), [list(r) for r in table], list(kv_len), page_tokens

    def _is(self, page):
        return 0 <= page < len(self.refs)

    def _pages(self, length):
        return -(-max(length, 0) // self.pt)

    def _held(self, b):
        return min(self._pages(self.kv_len[b]), len(self.table[b]))

    def _lowest(self):
        return next((i for i, r in enumerate(self.refs) if r <= 0), None)

    def _release(self, b):
        for j in range(self._held(b)):
            if self._is(self.table[b][j]):
                self.refs[self.table[b][j]] -= 1
            self.table[b][j] = -1
        self.kv_len[b] = 0

    def free(self, seqs):
        done = set()
        for b in seqs:
            if 0 <= b < len(self.kv_len) and b not in done:
                self._release(b)
                done.add(b)

    def extend(self, n_new):
        missing, short = [], False
        for b, n in enumerate(n_new):
            length, n = max(self.kv_len[b], 0), max(n, 0)
            have, want = self._pages(length), self._pages(length + n)
            if n > 0 and (want > len(self.table[b]) or length + n > 2 ** 31 - 1):
                missing.append(-1)
                continue
            if want > have and (short or sum(r <= 0 for r in self.refs) < want - have):
                short = True
                missing.append(want - have)
                continue
            for j in range(have, want):
                page = self._lowest()
                self.refs[page], self.table[b][j] = 1, page
            self.kv_len[b] = length + n
            missing.append(0)
        return missing

    def fork(self, src, dst):
        """Returns (status, copies), copies as (source page, new page, slots)."""
        status, tails = [], []
        for i, (s, t) in enumerate(zip(src, dst)):
            B = len(self.kv_len)
            if not (0 <= s < B and 0 <= t < B) or t in src or t in dst[:i]:
                status.append(-1)
                continue
            status.append(0)
            self._release(t)
            length = min(max(self.kv_len[s], 0), len(self.table[s]) * self.pt)
            full, tail = length // self.pt, length % self.pt
            for j in range(full):
                page = self.table[s][j]
                self.table[t][j] = page if self._is(page) else -1
                if self._is(page):
                    self.refs[page] += 1
            self.kv_len[t] = length
            if tail:
                self.table[t][full] = -1
                if self._is(self.table[s][full]):
                    self.kv_len[t] = full * self.pt
                    tails.append((i, s, t, full, tail))
        copies = []
        for i, s, t, full, tail in tails:  # pages are looked for when everything that goes back has gone
            page = self._lowest()
            if page is None:
                status[i] = 1
                continue
            self.refs[page], self.table[t][full] = 1, page
            self.kv_len[t] += tail
            copies.append((self.table[s][full], page, tail))
        return status, copies
