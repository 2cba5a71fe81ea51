"""Plain models, in 64 bits on the host, of the cut laws and of the cache's pages: what the GPU
tests compare with.  Each is the definition in the header, one row or one list entry at a time.

Every decision of a draw compares sums of float64 weights.  The model reports how near the nearest
of them was (relative to the row's sum), so that a test can require its inputs to be clear of the
rounding of either side: at most V additions of V terms with a relative error of a few 2^-53
each, below 1e-9 for V <= 2^20.
"""
from __future__ import annotations

import numpy as np

CLEAR = 1e-9


def law(x, T=1.0, k=0, p=1.0, m=0.0):
    """(probabilities float64, margin), or None for a row without a law."""
    x = np.asarray(x, np.float64) + 0.0
    V = len(x)
    T, p, m = float(T), float(p), float(m)
    if not (0 <= T < np.inf and 0 <= p <= 1 and 0 <= m <= 1):
        return None
    if np.isnan(x).any() or (x == np.inf).any() or not np.isfinite(x).any():
        return None
    if T == 0:
        T, k = 1.0, 1
    order = np.argsort(-x, kind="stable")
    if 0 < k < V:
        order = order[:k]
    w = np.exp((x[order] - x[order[0]]) / T)
    margin = np.inf
    if p < 1:
        run = np.concatenate([[0.0], np.cumsum(w)])
        total = run[-1]
        keep = run[:-1] < p * total
        keep[0] = True
        near = run[1:-1]
        # sums of equal weights 1 are exact on either side
        exact = (w[:-1] == 1.0) & (p * total == np.floor(p * total))
        gap = np.where(exact, np.inf, np.abs(near - p * total) / total)
        margin = min(margin, gap.min(initial=np.inf))
        order, w = order[keep], w[keep]
    if 0 < m < 1:
        margin = min(margin, np.abs(w - m).min())
    stay = w >= m
    out = np.zeros(V)
    out[order[stay]] = w[stay]
    return out / out.sum(), margin


def draw(w, u):
    """(id, margin): the first id whose inclusive prefix sum exceeds u times the sum."""
    c = np.cumsum(w)
    t = float(u) * c[-1]
    i = int(np.searchsorted(c, t, side="right"))
    pos = np.flatnonzero(w > 0)
    if i >= len(w):
        i = int(pos[-1])
    edges = c[pos]
    gap = np.abs(edges - t) / c[-1]
    if u == 0.0 or u == 1.0:
        return i, (np.inf if u == 0.0 else 0.0)
    return i, float(gap.min())


def sample(rows, u, T, k, p, m):
    """tokens, probabilities, margins of one draw per row."""
    n = len(rows)
    tok = np.full(n, -1, np.int64)
    prob = np.full(n, np.nan)
    mar = np.full(n, np.inf)
    for i in range(n):
        r = law(rows[i], T[i], int(k[i]), p[i], m[i])
        if r is None:
            continue
        tok[i], g = draw(r[0], u[i])
        prob[i] = r[0][tok[i]]
        mar[i] = min(g, r[1])
    return tok, prob, mar


def verify(tgt, drf, x, u, ft, fd):
    """accepted_len, tokens, probabilities, margins.  tgt [B][K+1][V], drf [B][K][V]; ft and fd are
    dicts of per-sequence parameters."""
    B, K1, V = tgt.shape
    K = K1 - 1
    acc = np.full(B, -1, np.int64)
    out = np.full((B, K + 1), -1, np.int64)
    prob = np.full((B, K, 2), np.nan)
    mar = np.full(B, np.inf)
    for b in range(B):
        par = lambda f: (f["T"][b], int(f["k"][b]), f["p"][b], f["m"][b])
        P = [law(tgt[b, j], *par(ft)) for j in range(K + 1)]
        Q = [law(drf[b, j], *par(fd)) for j in range(K)]
        if any(r is None for r in P + Q) or ((x[b] < 0) | (x[b] >= V)).any():
            continue
        mar[b] = min([r[1] for r in P + Q])
        L = None
        for j in range(K):
            pj, qj = P[j][0][x[b, j]], Q[j][0][x[b, j]]
            prob[b, j] = pj, qj
            if pj > 0 and qj > 0:
                mar[b] = min(mar[b], abs(float(u[b, j]) * qj - pj) / max(pj, qj))
            if L is None and not (pj > 0 and float(u[b, j]) * qj <= pj):
                L = j
        if L is None:
            L = K
            w = P[K][0]
        else:
            w = np.maximum(P[L][0] - Q[L][0], 0.0)
            if w.sum() == 0:
                w = P[L][0]
            else:
                # each p - q carries the rounding of p and q; relative to what is left of them
                mar[b] = min(mar[b], w.sum())
        acc[b] = L
        out[b, :L] = x[b, :L]
        out[b, L], g = draw(w, u[b, K])
        mar[b] = min(mar[b], g)
    return acc, out, prob, mar


class Pages:
    """A cache's books, one list entry after another."""

    def __init__(self, num_pages, page_tokens, num_seqs, max_blocks):
        self.pt, self.mb = page_tokens, max_blocks
        self.refs = [0] * num_pages
        self.rows = [[] for _ in range(num_seqs)]
        self.len = [0] * num_seqs
        self.moves = []              # (from, to) page copies of the last call

    def arrays(self):
        t = np.full((len(self.rows), self.mb), -1, np.int32)
        for i, r in enumerate(self.rows):
            t[i, :len(r)] = r
        return (np.array(self.refs, np.int32), t, np.array([len(r) for r in self.rows], np.int32),
                np.array(self.len, np.int32))

    def _free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def _firsts(self, seqs):
        seen, ok = set(), []
        for s in seqs:
            ok.append(0 <= s < len(self.rows) and s not in seen)
            seen.add(s)
        return ok

    def _grant(self, asks):
        free, total, places = self._free(), 0, []
        for a in asks:
            if a is None:
                places.append(None)
                continue
            total += a
            places.append(free[total - a:total] if total <= len(free) else None)
        return places

    def reserve(self, seqs, counts):
        before = list(self.refs)
        asks = []
        for s, c, ok in zip(seqs, counts, self._firsts(seqs)):
            if not ok or c < 0 or -(-(self.len[s] + c) // self.pt) > self.mb:
                asks.append(None)
                continue
            cow = c > 0 and self.len[s] % self.pt and before[self.rows[s][self.len[s] // self.pt]] > 1
            new = max(0, -(-(self.len[s] + c) // self.pt) - len(self.rows[s])) if c else 0
            asks.append(new + bool(cow))
        self.moves = []
        got = self._grant(asks)
        for s, c, g in zip(seqs, counts, got):
            if not g:
                continue
            g = list(g)
            at = self.len[s] // self.pt
            if self.len[s] % self.pt and before[self.rows[s][at]] > 1:
                new = g.pop(0)
                self.moves.append((self.rows[s][at], new))
                self.refs[self.rows[s][at]] -= 1
                self.refs[new] = 1
                self.rows[s][at] = new
            for pg in g:
                self.refs[pg] = 1
                self.rows[s].append(pg)
        return [-1 if g is None else 0 for g in got]

    def commit(self, seqs, accepted):
        status = []
        for s, a, ok in zip(seqs, accepted, self._firsts(seqs)):
            ok = ok and a >= -1 and self.len[s] + a + 1 <= len(self.rows[s]) * self.pt
            status.append(0 if ok else -1)
            if ok:
                self.len[s] += a + 1
                while len(self.rows[s]) > -(-self.len[s] // self.pt):
                    self.refs[self.rows[s].pop()] -= 1
        return status

    def fork(self, parents, children):
        n = len(self.rows)
        asks = []
        state = [(list(r), ln) for r, ln in zip(self.rows, self.len)]
        for a, b, ok in zip(parents, children, self._firsts(children)):
            ok = ok and 0 <= a < n and a != b and not state[b][0] and state[b][1] == 0
            asks.append(int(state[a][1] % self.pt != 0) if ok else None)
        got = self._grant(asks)
        self.moves = []
        for a, b, g in zip(parents, children, got):
            if g is None:
                continue
            row, ln = state[a]
            row = row[:-(-ln // self.pt)]
            if g:
                self.moves.append((row[-1], g[0]))
                row = row[:-1] + [g[0]]
            for pg in row:
                self.refs[pg] += 1
            self.rows[b], self.len[b] = row, ln
        return [-1 if g is None else 0 for g in got]

    def free(self, seqs, keep=None):
        for i, s in enumerate(seqs):
            if (keep is None or not keep[i]) and 0 <= s < len(self.rows):
                for pg in self.rows[s]:
                    self.refs[pg] -= 1
                self.rows[s], self.len[s] = [], 0

    def compact(self):
        used = [p for p, r in enumerate(self.refs) if r > 0]
        U = len(used)
        to = {p: p for p in used}
        holes = [p for p in range(U) if self.refs[p] == 0]
        self.moves = list(zip([p for p in used if p >= U], holes))
        for a, b in self.moves:
            to[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.rows = [[to[p] for p in r] for r in self.rows]
        return [to.get(p, -1) for p in range(len(self.refs))], U
