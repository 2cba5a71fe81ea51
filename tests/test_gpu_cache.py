"""The cache's pages on the GPU against the sequential model: state, statuses and page contents
are integers and copies, so everything is equal."""
import numpy as np
import pytest
import torch

import filter_model as model
from gpu_support import dev
from rejection_sampling_verification_row_amd import binding as sv

pytestmark = pytest.mark.gpu


class Cache:
    """A handle with its state and pools on the GPU, and the model beside it."""

    def __init__(self, pages, pt, seqs, blocks, pools=2, page_bytes=48, seed=0):
        self.m = model.Pages(pages, pt, seqs, blocks)
        self.pages, self.n = pages, seqs
        self.state = [dev(a) for a in self.m.arrays()]
        r = np.random.RandomState(seed)
        self.data = [r.randint(0, 256, (pages, page_bytes)).astype(np.uint8) for _ in range(pools)]
        self.pools = [dev(d) for d in self.data]
        self.h = sv.specverify_cache_create(0, pages, pt, seqs, blocks, page_bytes, self.pools,
                                            *self.state)

    def load(self):
        """The model's books into the device state."""
        for s, a in zip(self.state, self.m.arrays()):
            s.copy_(dev(a))

    def check(self, moves=True):
        torch.cuda.synchronize()
        for name, s, a in zip(("refs", "tables", "blocks", "lengths"), self.state, self.m.arrays()):
            assert np.array_equal(s.cpu().numpy(), a), name
        if moves:
            for d in self.data:
                for a, b in self.m.moves:
                    d[b] = d[a]
            self.m.moves = []
        for p, d in zip(self.pools, self.data):
            assert np.array_equal(p.cpu().numpy(), d)

    def call(self, op, *lists, stream=None):
        arrays = [None if a is None else dev(np.asarray(a, np.int32)) for a in lists]
        n = len(lists[-1])
        status = torch.full((n,), -7, dtype=torch.int32, device="cuda")
        getattr(sv, "specverify_cache_" + op)(self.h, stream, n, *arrays, status)
        first = range(n) if lists[0] is None else lists[0]
        want = getattr(self.m, op)(first, *lists[1:])
        self.check()
        assert status.tolist() == want
        return want

    def free(self, seqs, keep=None):
        n = self.n if seqs is None else len(seqs)
        sv.specverify_cache_free(self.h, None, n, None if seqs is None else dev(np.asarray(seqs, np.int32)),
                                 None if keep is None else dev(np.asarray(keep, np.uint8)))
        self.m.free(range(n) if seqs is None else seqs, keep)
        self.check()

    def compact(self):
        pm = torch.full((self.pages,), -7, dtype=torch.int32, device="cuda")
        used = torch.zeros(1, dtype=torch.int32, device="cuda")
        sv.specverify_cache_compact(self.h, None, pm, used)
        to, U = self.m.compact()
        self.check()
        assert pm.tolist() == to and used.item() == U

    def __del__(self):
        sv.specverify_cache_destroy(self.h)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("pages,pt,seqs,blocks,pools,page_bytes", [
    (40, 4, 10, 8, 2, 48), (1, 1, 2, 3, 1, 16), (300, 1, 33, 40, 3, 16), (5000, 16, 70, 100, 1, 256),
    (97, 7, 12, 20, 0, 0), (64, 3, 9, 9, 2, 16400), (64, 8, 9, 9, 1, 65536)])
def test_runs_of_random_calls(pages, pt, seqs, blocks, pools, page_bytes, seed):
    """Any calls in any order, refused entries, lists with repeats and full pools among them."""
    r = np.random.RandomState(seed)
    c = Cache(pages, pt, seqs, blocks, pools, page_bytes, seed)
    seen = set()
    for _ in range(40):
        n = r.randint(1, seqs + 1)
        s = r.randint(-1, seqs + 1, n) if r.rand() < 0.5 else r.permutation(seqs)[:n]
        op = r.choice(["reserve", "reserve", "commit", "fork", "free", "compact"])
        if op == "reserve":
            st = c.call(op, s, r.randint(-1, 3 * pt + 2, n))
        elif op == "commit":
            st = c.call(op, s, r.randint(-2, 2 * pt + 1, n))
        elif op == "fork":
            st = c.call(op, s, r.randint(-1, seqs + 1, n))
        elif op == "free":
            c.free(s, r.randint(0, 2, n))
            st = []
        else:
            c.compact()
            st = []
        seen.update((op, x) for x in st)
    if pages > 1:                # a pool of one page hardly lets a commit through
        assert {("reserve", 0), ("reserve", -1), ("commit", 0), ("commit", -1)} <= seen


def test_lists_longer_than_a_workgroup():
    """Thousands of entries and pages: the plan's scans run over many tiles."""
    r = np.random.RandomState(1)
    c = Cache(30000, 2, 2500, 30, 1, 16)
    c.call("reserve", None, r.randint(0, 20, 2500))
    c.call("commit", None, r.randint(-1, 12, 2500))
    c.call("fork", r.randint(0, 2500, 1200), r.permutation(2500)[:1200])
    c.free(r.permutation(2500)[:1300])
    c.call("fork", r.randint(0, 2500, 1300), r.permutation(2500)[:1300])
    c.compact()
    c.call("reserve", r.permutation(2500), r.randint(0, 25, 2500))


def test_a_pool_that_runs_out_refuses_from_there_on():
    c = Cache(10, 4, 6, 8)
    assert c.call("reserve", None, [12, 12, 12, 12, 0, 4]) == [0, 0, 0, -1, -1, -1]
    assert c.call("reserve", [5, 4], [4, 4]) == [0, -1]


def test_a_shared_partly_filled_page_is_copied_for_each_writer():
    c = Cache(12, 4, 4, 4)
    c.call("reserve", [0], [8])
    c.call("commit", [0], [7])
    c.call("fork", [0, 0], [1, 2])
    # cut back into the second, full and shared page
    for s in range(3):
        c.m.len[s] = 6
    c.load()
    c.call("reserve", [2, 0, 3], [1, 5, 0])
    c.call("reserve", [1], [0])                    # nothing to write: nothing copied
    c.call("reserve", [1], [1])                    # the last holder keeps the page


def test_contradicting_states_are_refused_and_bad_page_ids_skipped():
    c = Cache(8, 4, 6, 4)
    c.call("reserve", [0, 1], [6, 6])
    c.call("commit", [0, 1], [5, 5])
    refs, tables, blocks, lengths = c.state
    blocks[2], lengths[2] = 2, 9                   # more tokens than its pages hold
    blocks[3] = 5                                  # more blocks than a table has
    lengths[4] = -1
    tables[1, 1] = 99
    before = [s.clone() for s in c.state]
    st = torch.zeros(3, dtype=torch.int32, device="cuda")
    bad = dev(np.array([2, 3, 4], np.int32))
    for fn, arg in ((sv.specverify_cache_reserve, 1), (sv.specverify_cache_commit, -1)):
        fn(c.h, None, 3, bad, torch.full((3,), arg, dtype=torch.int32, device="cuda"), st)
        assert st.tolist() == [-1, -1, -1]
    sv.specverify_cache_fork(c.h, None, 3, bad, dev(np.array([5, 5, 5], np.int32)), st)
    assert st.tolist() == [-1, -1, -1]
    for a, b in zip(before, c.state):
        assert torch.equal(a, b)
    # sequence 1's second page id, 3, was overwritten with one out of range: that entry's release
    # is left out, and page 3 keeps its count
    one = dev(np.array([1], np.int32))
    sv.specverify_cache_reserve(c.h, None, 1, one, one, st)
    sv.specverify_cache_free(c.h, None, 1, one, None)
    torch.cuda.synchronize()
    assert refs.tolist() == [1, 1, 0, 1, 0, 0, 0, 0] and blocks[1] == 0
    for p, d in zip(c.pools, c.data):
        assert np.array_equal(p.cpu().numpy(), d)


def test_copy_and_what_it_refuses():
    c = Cache(20, 4, 2, 4, 3, 4096 + 16)
    src = [0, 1, 2, 3, 4, 5, 20, -1, 7, 6, 10]
    dst = [10, 11, 11, 12, 20, -2, 13, 14, 7, 15, 16]
    status = torch.full((11,), -7, dtype=torch.int32, device="cuda")
    sv.specverify_cache_copy(c.h, None, 11, dev(np.array(src, np.int32)),
                             dev(np.array(dst, np.int32)), status)
    torch.cuda.synchronize()
    # 2: second to name page 11; 7: its own source; 10 reads what entry 0 writes
    assert status.tolist() == [0, 0, -1, 0, -1, -1, -1, -1, -1, 0, -1]
    c.m.moves = [(0, 10), (1, 11), (3, 12), (6, 15)]
    c.check()
    # the marks of the last call are gone
    sv.specverify_cache_copy(c.h, None, 1, dev(np.array([10], np.int32)),
                             dev(np.array([2], np.int32)), status)
    c.m.moves = [(10, 2)]
    c.check()
    assert status[0] == 0


def test_offsets_past_32_bits():
    """Page 70000 of 64 KiB pages lies past 4 GiB of its pool."""
    pool = torch.zeros(70016, 65536, dtype=torch.uint8, device="cuda")
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    refs, tables, blocks, lengths = ints(70016), ints(2, 2), ints(2), ints(2)
    refs[:70000] = 1
    tables.fill_(-1)
    h = sv.specverify_cache_create(0, 70016, 16, 2, 2, 65536, [pool], refs, tables, blocks, lengths)
    pool[65537] = torch.randint(0, 256, (65536,), dtype=torch.uint8, device="cuda")
    sv.specverify_cache_copy(h, None, 1, dev(np.array([65537], np.int32)),
                             dev(np.array([70001], np.int32)))
    sv.specverify_cache_reserve(h, None, 1, None, dev(np.array([17], np.int32)))
    torch.cuda.synchronize()
    assert torch.equal(pool[70001], pool[65537]) and tables[0].tolist() == [70000, 70001]
    assert pool[65537 - 65536].sum() == 0        # where a wrapped offset would have written
    sv.specverify_cache_destroy(h)


def test_argument_errors():
    c = Cache(8, 4, 3, 4)
    i = torch.zeros(9, dtype=torch.int32, device="cuda")

    def status(fn, *a):
        with pytest.raises(sv.SpecVerifyError) as e:
            fn(c.h, None, *a)
        return e.value.status

    for fn in (sv.specverify_cache_reserve, sv.specverify_cache_commit, sv.specverify_cache_fork):
        assert status(fn, 4, i, i, i) == sv.SPECVERIFY_ECAPACITY
        assert status(fn, -1, i, i, i) == sv.SPECVERIFY_EINVAL
        assert status(fn, 1, i, None, i) == sv.SPECVERIFY_EINVAL
        assert status(fn, 1, i, i.data_ptr() + 2, i) == sv.SPECVERIFY_EINVAL
        fn(c.h, None, 0, None, None, None)
    assert status(sv.specverify_cache_fork, 1, None, i, i) == sv.SPECVERIFY_EINVAL
    assert status(sv.specverify_cache_copy, 9, i, i, i) == sv.SPECVERIFY_ECAPACITY
    assert status(sv.specverify_cache_copy, 1, None, i, i) == sv.SPECVERIFY_EINVAL
    assert status(sv.specverify_cache_free, 4, i) == sv.SPECVERIFY_ECAPACITY
    assert status(sv.specverify_cache_compact, i.data_ptr() + 1) == sv.SPECVERIFY_EINVAL
    with pytest.raises(ValueError):
        sv.specverify_cache_compact(c.h, None, i[:7])          # a map of 8 pages
    assert sv.specverify_cache_workspace_bytes(c.h) > 0
    c.check()


def test_replays_of_a_captured_step():
    """Reserve and commit captured once, replayed with new lists and eager work between: each
    replay moves the state on as the model says."""
    c = Cache(400, 4, 24, 16, 2, 1024)
    counts, acc = (torch.zeros(24, dtype=torch.int32, device="cuda") for _ in range(2))
    status = torch.zeros(2, 24, dtype=torch.int32, device="cuda")

    def go():
        sv.specverify_cache_reserve(c.h, None, 24, None, counts, status[0])
        sv.specverify_cache_commit(c.h, None, 24, None, acc, status[1])

    acc.fill_(-1)
    go()                                        # a step that changes nothing
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    r = np.random.RandomState(3)
    for step in range(5):
        k, a = r.randint(0, 6, 24), r.randint(-1, 5, 24)
        counts.copy_(dev(k.astype(np.int32)))
        acc.copy_(dev(a.astype(np.int32)))
        graph.replay()
        s0 = c.m.reserve(range(24), k)
        for d in c.data:
            for x, y in c.m.moves:
                d[y] = d[x]
        c.m.moves = []
        s1 = c.m.commit(range(24), a)
        c.check()
        assert status.tolist() == [s0, s1]
        if step == 2:                           # eager calls between the replays
            c.free([0, 1, 2])
            c.call("fork", [5, 6], [0, 2])


def test_another_stream():
    c = Cache(64, 4, 8, 8)
    st = torch.cuda.Stream()
    counts, taken = dev(np.full(8, 9, np.int32)), dev(np.arange(8, dtype=np.int32))
    torch.cuda.synchronize()
    sv.specverify_cache_reserve(c.h, st, 8, None, counts)
    sv.specverify_cache_commit(c.h, st, 8, None, taken)
    st.synchronize()
    c.m.reserve(range(8), [9] * 8)
    c.m.commit(range(8), list(range(8)))
    c.check()


def test_a_served_round_of_the_operators_together():
    """Best-of-N over one prompt each: fork the candidates, draft with the cut sampler, make room,
    verify with the same cuts, commit what was accepted, cut the candidates by reward, free the
    rest, compact: every step reads what the one before wrote, on one stream, with no copy back."""
    P, N, K, V = 3, 4, 3, 2003
    B = P * N
    r = np.random.RandomState(2)
    c = Cache(200, 4, P + B, 12, 2, 512)
    prompts = list(range(P))
    c.call("reserve", prompts, [9, 16, 6])
    c.call("commit", prompts, [8, 15, 5])
    kids = np.arange(P, P + B).astype(np.int32)
    parents = np.repeat(np.arange(P), N).astype(np.int32)
    q = dict(T=np.full(B, 0.9, np.float32), k=np.full(B, 30, np.int32),
             p=np.full(B, 0.95, np.float32), m=np.full(B, 0.01, np.float32))
    f = sv.SpecVerifyFilter(temperature=dev(q["T"]), top_k=dev(q["k"]), top_p=dev(q["p"]),
                            min_p=dev(q["m"]))
    tgt = (r.standard_normal((B, K + 1, V)) * 3).astype(np.float32)
    drf = tgt[:, :K] + r.standard_normal((B, K, V)).astype(np.float32) * 0.5
    ud, uv = r.rand(K, B).astype(np.float32), r.rand(B, K + 1).astype(np.float32)
    scores = r.standard_normal((P, N)).astype(np.float32)
    ctx = sv.specverify_create(0, B, K, V)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    dt, dd = dev(tgt), dev(drf)
    col, tokens, acc, out = i32(B), i32(B, K), i32(B), i32(B, K + 1)
    keep, cut, nk = torch.zeros(P, N, dtype=torch.uint8, device="cuda"), torch.zeros(P, device="cuda"), i32(P)
    dk, dp = dev(kids), dev(parents)
    sv.specverify_cache_fork(c.h, None, B, dp, dk)
    for j in range(K):
        sv.specverify_sample_filtered(ctx, None, sv.SPECVERIFY_F32, B, V, K * V, f,
                                      dd.data_ptr() + 4 * j * V, dev(ud[j]), col)
        tokens[:, j] = col
    sv.specverify_cache_reserve(c.h, None, B, dk, torch.full((B,), K + 1, dtype=torch.int32, device="cuda"))
    sv.specverify_run_sampling_filtered(ctx, None, sv.SPECVERIFY_F32, B, K, V, f, None, dt, dd,
                                        tokens, dev(uv), acc, out)
    sv.specverify_cache_commit(c.h, None, B, dk, acc)
    sv.specverify_quantile_cut(ctx, None, P, N, 0.5, dev(scores), cut, keep, nk)
    sv.specverify_cache_free(c.h, None, B, dk, keep)
    torch.cuda.synchronize()
    # the same by the models
    x = np.zeros((B, K), np.int32)
    for j in range(K):
        x[:, j] = model.sample(drf[:, j], ud[j], q["T"], q["k"], q["p"], q["m"])[0]
    a, o, _, mar = model.verify(tgt, drf, x, uv, q, q)
    assert np.all(mar > model.CLEAR)
    assert np.array_equal(tokens.cpu().numpy(), x) and np.array_equal(acc.cpu().numpy(), a)
    assert np.array_equal(out.cpu().numpy(), o)
    kept = scores >= np.sort(scores, axis=1)[:, 2:3]
    assert np.array_equal(keep.cpu().numpy().astype(bool), kept)
    mv = []
    c.m.fork(parents, kids)
    mv += c.m.moves
    c.m.reserve(kids, [K + 1] * B)
    mv += c.m.moves
    c.m.commit(kids, a)
    c.m.free(kids, kept.reshape(-1))
    c.m.moves = mv
    c.check()
    c.compact()
    sv.specverify_destroy(ctx)


def test_a_pool_of_millions_of_pages():
    """More stretches of the pool than a plan keeps in LDS, with few pages free among them."""
    pages, seqs, blocks = 4096 * 1100 + 77, 40, 300
    r = np.random.RandomState(8)
    refs = np.ones(pages, np.int32)
    free = np.sort(r.permutation(pages)[:9000]).astype(np.int32)
    refs[free] = 0
    dr = dev(refs)
    tables = torch.full((seqs, blocks), -1, dtype=torch.int32, device="cuda")
    zero = lambda: torch.zeros(seqs, dtype=torch.int32, device="cuda")
    bl, ln, st = zero(), zero(), zero()
    h = sv.specverify_cache_create(0, pages, 1, seqs, blocks, 0, [], dr, tables, bl, ln)
    counts = r.randint(0, 300, seqs).astype(np.int32)
    sv.specverify_cache_reserve(h, None, seqs, None, dev(counts), st)
    torch.cuda.synchronize()
    upto = np.cumsum(counts)
    assert upto[-1] <= 9000 and st.tolist() == [0] * seqs and bl.tolist() == counts.tolist()
    t = tables.cpu().numpy()
    for i in range(seqs):
        assert np.array_equal(t[i, :counts[i]], free[upto[i] - counts[i]: upto[i]])
        assert np.all(t[i, counts[i]:] == -1)
    refs[free[:upto[-1]]] = 1
    assert np.array_equal(dr.cpu().numpy(), refs)
    pm = torch.zeros(pages, dtype=torch.int32, device="cuda")
    used = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.specverify_cache_compact(h, None, pm, used)
    torch.cuda.synchronize()
    U = int((refs > 0).sum())
    at = np.flatnonzero(refs > 0)
    want = np.full(pages, -1, np.int64)
    want[at] = at
    want[at[at >= U]] = np.flatnonzero(refs == 0)[:(at >= U).sum()]
    assert used.item() == U and np.array_equal(pm.cpu().numpy(), want)
    for i in range(seqs):
        assert np.array_equal(tables[i, :counts[i]].cpu().numpy(), want[t[i, :counts[i]]])
    sv.specverify_cache_destroy(h)


@pytest.mark.parametrize("pools,page_bytes", [(70, 32), (3, 33 * 16384 + 16), (1, 16 << 20)])
def test_pages_and_pools_of_many_sizes_are_copied_whole(pools, page_bytes):
    c = Cache(12, 4, 8, 3, pools, page_bytes)
    c.call("reserve", [0, 1], [6, 7])
    c.call("commit", [0, 1], [5, 6])
    c.call("fork", [0, 1, 0], [2, 3, 4])
    c.free([0, 3])
    c.compact()
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    sv.specverify_cache_copy(c.h, None, 2, dev(np.array([0, 1], np.int32)), dev(np.array([11, 10], np.int32)), status)
    c.m.moves = [(0, 11), (1, 10)]
    c.check()
