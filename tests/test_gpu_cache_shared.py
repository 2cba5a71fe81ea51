"""Reserve where a sequence's tokens were cut back past a page's edge: whatever it is going to write
into has no other holder afterwards."""
import numpy as np
import pytest

import filter_model as model
from test_gpu_cache import Cache

pytestmark = pytest.mark.gpu


class Pages(model.Pages):
    """The books with every shared page that a reserve gives room in replaced, not the partly filled
    one alone."""

    def reserve(self, seqs, counts):
        before, pt = list(self.refs), self.pt
        asks, shared = [], []
        for s, c, ok in zip(seqs, counts, self._firsts(seqs)):
            shared.append([])
            if not ok or c < 0 or -(-(self.len[s] + c) // pt) > self.mb:
                asks.append(None)
                continue
            need = -(-(self.len[s] + c) // pt) if c else 0
            shared[-1] = [j for j in range(self.len[s] // pt, min(need, len(self.rows[s])))
                          if before[self.rows[s][j]] > 1]
            asks.append(len(shared[-1]) + max(0, need - len(self.rows[s])))
        self.moves = []
        got = self._grant(asks)
        for s, js, g in zip(seqs, shared, got):
            g = list(g or [])
            for j in js if g else []:
                old, new = self.rows[s][j], g.pop(0)
                if j * self.pt < self.len[s]:
                    self.moves.append((old, new))
                self.refs[old] -= 1
                self.refs[new] = 1
                self.rows[s][j] = new
            for pg in g:
                self.refs[pg] = 1
                self.rows[s].append(pg)
        return [-1 if g is None else 0 for g in got]


def cache(*a, **kw):
    c = Cache(*a, **kw)
    c.m.__class__ = Pages
    return c


def alone(c, seq, count):
    """The pages that hold tokens len .. len + count - 1 have one holder."""
    at = range(c.m.len[seq] // c.m.pt, -(-(c.m.len[seq] + count) // c.m.pt) if count else 0)
    refs, tables = c.state[0].cpu().numpy(), c.state[1].cpu().numpy()
    assert all(refs[tables[seq, j]] == 1 for j in at)


@pytest.mark.parametrize("length", [8, 7, 5, 4, 3, 2, 1, 0])
def test_a_sequence_cut_back_by_any_length_gets_pages_of_its_own(length):
    c = cache(24, 4, 4, 8)
    c.call("reserve", [0], [12])
    c.call("commit", [0], [11])
    c.call("fork", [0, 0], [1, 2])
    c.m.len[0] = c.m.len[2] = length
    c.load()
    kept = c.pools[0][c.state[1][1, :3].long()].cpu()
    assert c.call("reserve", [0, 3, 2], [4, 5, 9]) == [0, 0, 0]
    alone(c, 0, 4)
    alone(c, 2, 9)
    assert (c.pools[0][c.state[1][1, :3].long()].cpu() == kept).all()     # the other's are untouched
    c.call("commit", [0, 2], [3, 8])
    c.free(None)
    assert not c.state[0].any()


def test_replaced_pages_count_against_the_free_ones():
    c = cache(7, 4, 3, 8)
    c.call("reserve", [0], [16])
    c.call("commit", [0], [15])
    c.call("fork", [0], [1])
    c.m.len[0] = 2
    c.load()
    assert c.call("reserve", [0], [14]) == [-1]            # four pages, three free
    assert c.call("reserve", [0, 2], [10, 1]) == [0, -1]   # three
    alone(c, 0, 10)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("pages,pt,seqs,blocks", [(60, 4, 10, 8), (3000, 1, 33, 150), (16000, 3, 1100, 12)])
def test_runs_of_calls_with_lengths_cut_back_between(pages, pt, seqs, blocks, seed):
    r = np.random.RandomState(seed)
    c = cache(pages, pt, seqs, blocks, 2, 32, seed)
    replaced = 0
    for _ in range(10):
        # some grow by what they reserve, some empty ones become copies, some are cut back
        n = r.randint(1, seqs + 1)
        s = r.permutation(seqs)[:n]
        counts = r.randint(1, blocks * pt // 2 + 2, n)
        c.call("reserve", s, counts)
        c.call("commit", s, counts - 1)
        c.free(r.permutation(seqs)[:seqs // 2])
        c.call("fork", r.randint(0, seqs, seqs), r.permutation(seqs))
        for i in range(seqs):
            if r.rand() < 0.5:
                c.m.len[i] = r.randint(0, c.m.len[i] + 1)
        c.load()
        s = r.permutation(seqs)[:n]
        counts = r.randint(0, blocks * pt // 2 + 2, n)
        held = [list(c.m.rows[i]) for i in s]
        for i, k, st, h in zip(s, counts, c.call("reserve", s, counts), held):
            if st == 0:
                alone(c, i, k)
                first = -(-c.m.len[i] // pt)
                replaced += h[first:] != c.m.rows[i][first:len(h)]
        c.call("commit", s, r.randint(-1, pt + 1, n))
    assert replaced > 2
