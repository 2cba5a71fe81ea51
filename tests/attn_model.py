"""Models in 64 bits of the attention over a cache, its append, the tree verify and the path's move:
written from the definitions in the header, node by node."""
import numpy as np


def depths(parents, count):
    """Depth of each node (parents: a list, None for a chain), None if one is not below its child."""
    d = []
    for t in range(count):
        p = t - 1 if parents is None else int(parents[t])
        if t and not 0 <= p < t:
            return None
        d.append(d[p] + 1 if t else 0)
    return d


def sees(parents, t):
    """Node t and its ancestors, nearest first."""
    out = [t]
    while t:
        t = t - 1 if parents is None else int(parents[t])
        out.append(t)
    return out


def rotate(x, pos, inv_freq, dims, inter):
    """x [heads, D] float64 at position pos."""
    y = x.copy()
    if not dims:
        return y
    half = dims // 2
    f = float(pos) * inv_freq.astype(np.float64)[:half]
    c, s = np.cos(f), np.sin(f)
    a, b = (x[:, 0:dims:2], x[:, 1:dims:2]) if inter else (x[:, :half], x[:, half:dims])
    u, v = a * c - b * s, b * c + a * s
    if inter:
        y[:, 0:dims:2], y[:, 1:dims:2] = u, v
    else:
        y[:, :half], y[:, half:dims] = u, v
    return y


class Step:
    """What the calls of one step are given: the cache's state as arrays, entries and nodes."""

    def __init__(self, pt, num_pages, tables, blocks, lengths, n, max_count, rows, seqs=None, starts=None,
                 counts=None, parents=None):
        self.__dict__.update(locals())
        del self.__dict__["self"]

    def entry(self, i, once=False):
        """(sequence, start, count, length, parents) of entry i, None if it is refused."""
        s = i if self.seqs is None else int(self.seqs[i])
        a = i * self.max_count if self.starts is None else int(self.starts[i])
        m = self.max_count if self.counts is None else int(self.counts[i])
        if not 0 <= s < len(self.blocks):
            return None
        b, ln = int(self.blocks[s]), int(self.lengths[s])
        if not 0 <= b <= self.tables.shape[1] or not 0 <= ln <= b * self.pt:
            return None
        if not 0 <= m <= self.max_count or ln + m > b * self.pt or a < 0 or a + m > self.rows:
            return None
        par = None if self.parents is None else [int(p) for p in self.parents[a:a + m]]
        if depths(par, m) is None:
            return None
        if once and self.seqs is not None and s in [int(x) for x in self.seqs[:i]]:
            return None
        return s, a, m, ln, par

    def slot(self, s, j):
        """Place of token j of sequence s in a pool, None without a page."""
        p = int(self.tables[s, j // self.pt])
        return p * self.pt + j % self.pt if 0 <= p < self.num_pages else None


def append(st, kpool, vpool, k, v, q, inv_freq, dims, inter):
    """Writes into kpool, vpool [slots, heads, D] and returns rotated queries (q where there is
    nothing) and statuses.  All float64."""
    status, out = [], None if q is None else q.copy()
    for i in range(st.n):
        e = st.entry(i, once=True)
        status.append(-1 if e is None else 0)
        if e is None:
            continue
        s, a, m, ln, par = e
        d = depths(par, m)
        for t in range(m):
            if q is not None:
                out[a + t] = rotate(q[a + t], ln + d[t], inv_freq, dims, inter)
            at = st.slot(s, ln + t)
            if at is not None:
                kpool[at] = rotate(k[a + t], ln + d[t], inv_freq, dims, inter)
                vpool[at] = v[a + t]
    return out, status


def attend(st, kpool, vpool, q, scale, window, kv_heads):
    """(out [rows, H, D], lse [rows, H], statuses, rows written, weight of |v| per row): float64; rows
    that no entry has are NaN."""
    H, D = q.shape[1:]
    G = H // kv_heads
    out = np.full(q.shape, np.nan)
    size = np.full(q.shape, np.nan)
    lse = np.full(q.shape[:2], np.nan)
    status, rows = [], []
    for i in range(st.n):
        e = st.entry(i)
        status.append(-1 if e is None else 0)
        if e is None:
            continue
        s, a, m, ln, par = e
        d = depths(par, m)
        for t in range(m):
            low = max(0, ln + d[t] - window + 1) if window else 0
            js = list(range(low, ln)) + [ln + b for b in sees(par, t) if not window or d[t] - d[b] < window]
            at = [x for x in (st.slot(s, j) for j in sorted(js)) if x is not None]
            rows.append(a + t)
            for h in range(H):
                kk, vv = kpool[at, h // G], vpool[at, h // G]
                with np.errstate(invalid="ignore"):
                    x = scale * (kk @ q[a + t, h]) if at else np.zeros(0)
                if not at or np.all(x == -np.inf):
                    out[a + t, h], lse[a + t, h], size[a + t, h] = 0, -np.inf, 0
                    continue
                with np.errstate(all="ignore"):
                    top = x.max()
                    w = np.exp(x - top)
                    z = w.sum()
                    out[a + t, h] = (w[:, None] * vv).sum(0) / z
                    size[a + t, h] = (w[:, None] * np.abs(vv)).sum(0) / z
                    lse[a + t, h] = top + np.log(z)
    return out, lse, status, rows, size


def walk(best, tokens, parents, count, T, V, depth):
    """(accepted, path, tokens) of one tree, from its rows' best ids."""
    bad = (-1, [-1] * (depth + 1), [-1] * (depth + 1))
    if not 1 <= count <= T:
        return bad
    for i in range(1, count):
        if not 0 <= tokens[i] < V or not 0 <= parents[i] < i:
            return bad
    at, path, out = 0, [], []
    while True:
        path.append(at)
        out.append(int(best[at]))
        nxt = [i for i in range(1, count) if parents[i] == at and tokens[i] == best[at]]
        if not nxt or len(path) > depth:
            break
        at = nxt[0]
    fill = [-1] * (depth + 1 - len(path))
    return len(path) - 1, path + fill, out + fill


def keep_path(pt, num_pages, tables, blocks, lengths, pools, n, max_count, seqs, accepted, path):
    """Moves tokens of pools [pool][slots, bytes]; statuses."""
    status = []
    for i in range(n):
        s, L = (i if seqs is None else int(seqs[i])), int(accepted[i])
        ok = 0 <= s < len(blocks) and -1 <= L < max_count
        ok = ok and not (seqs is not None and s in [int(x) for x in seqs[:i]])
        if ok:
            b, ln = int(blocks[s]), int(lengths[s])
            ok = 0 <= b <= tables.shape[1] and 0 <= ln <= b * pt
        if ok and L >= 0:
            p = [int(x) for x in path[i, :L + 1]]
            ok = p[0] == 0 and all(x < y for x, y in zip(p, p[1:])) and ln + p[-1] < b * pt
        status.append(0 if ok else -1)
        if not ok:
            continue
        for j in range(1, L + 1):
            ids = [int(tables[s, (ln + x) // pt]) for x in (p[j], j)]
            if all(0 <= x < num_pages for x in ids):
                src, dst = (g * pt + (ln + x) % pt for g, x in zip(ids, (p[j], j)))
                for pool in pools:
                    pool[dst] = pool[src]
    return status
