"""Attention over a paged cache in every form that the number of rows of a key head selects, over more
tokens than are under way at once, and the tree calls in a replayed graph.  Bounds are those of
test_gpu_attn."""
import numpy as np
import pytest
import torch

from gpu_support import dev
from rejection_sampling_verification_row_amd import binding as sv
from test_gpu_attn import TD, Setup
from test_gpu_tree import I32, Books, forest, paths

pytestmark = pytest.mark.gpu

# query heads of a key head and nodes: 16 rows and fewer, then one and all of each form's rows and more
ROWS = [(4, 4), (1, 17), (4, 8), (3, 11), (8, 8), (5, 13), (16, 8), (43, 3), (8, 32), (5, 60)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 72, 128, 256])
@pytest.mark.parametrize("group,m", ROWS)
def test_forms_over_many_tokens(dt, D, group, m):
    s = Setup(dt, group, 1, D, 16, [1500, 129, 0, 700], [m, 1, m, max(m - 1, 1)], seed=m + D)
    s.device().check_attend()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group,m", [(4, 4), (4, 8), (8, 8), (16, 8), (8, 32)])
@pytest.mark.parametrize("down", [False, True])
def test_forms_whose_maxima_grow(dt, D, group, m, down):
    """Keys that grow along the sequence, or shrink: the running maximum is left behind again and
    again, or never."""
    Hk = 2 if group == 4 else 1
    s = Setup(dt, Hk * group, Hk, D, 16, [900], [m], seed=D)
    st = s.step()
    q = st.entry(0)[0]
    t, f = s.pools[0]
    flat, flat64 = t.view(-1, s.Hk, D), f.reshape(-1, s.Hk, D)
    for j in range(900):
        at = st.slot(q, j)
        flat[at] = (flat[at].float() * ((900 - j if down else j) / 300)).to(TD[dt])
        flat64[at] = flat[at].double().numpy()
    s.device().check_attend()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 80, 128, 256])
@pytest.mark.parametrize("group,m", [(4, 4), (2, 12), (4, 12), (8, 12), (16, 12), (32, 12)])
def test_odd_values_and_lost_pages_in_every_form(dt, D, group, m):
    """NaN and infinities in nodes that their siblings do not see, and pages that are not there."""
    s = Setup(dt, group, 1, D, 8, [700, 90, 5], [m, m, 3], seed=7)
    r = np.random.RandomState(D)
    st = s.step()
    for i, odd in enumerate((np.nan, np.inf, -np.inf)):
        q, a, c, ln, par = st.entry(i)
        at = st.slot(q, ln + c - 1)
        for t, f in s.pools:
            f.reshape(-1, 1, D)[at, :, r.randint(0, D, 3)] = odd
            t.view(-1, 1, D)[at] = torch.from_numpy(f.reshape(-1, 1, D)[at]).to(TD[dt])
        if i == 0:
            for b in (3, 40):
                page = s.tables[q, b]
                for t, f in s.pools:
                    f[page] = odd
                    t[page] = odd
                s.tables[q, b] = (-1, s.P)[b == 40]
    s.device().check_attend()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_split_rows_are_joined(dt, D):
    """More rows than have a workgroup each in the join, most of segments that are split."""
    r = np.random.RandomState(D)
    lens, counts = r.randint(300, 1500, 26).tolist(), r.randint(1, 5, 26).tolist()
    Setup(dt, 32, 2, D, 16, lens, counts, seed=1).device().check_attend()


def test_tree_and_path_calls_on_a_stream_and_in_a_replayed_graph():
    """The three ways of the tree's walk and a path's move, captured once, replayed with other inputs."""
    r = np.random.RandomState(5)
    for B, T, V, depth in ((3, 12, 900, 4), (5, 33, 9000, 6), (96, 64, 32000, 3)):
        ctx = sv.specverify_create(0, B, T - 1, V)
        n = min(B, 8)
        books = Books(8, list(r.randint(0, 40, n)), [T] * n, 64, 2, seed=B)
        state = [dev(a) for a in (books.refs, books.tables, books.blocks, books.lengths)]
        pools = [dev(p) for p in books.pools]
        cache = sv.specverify_cache_create(0, books.P, 8, books.S, books.mb, 64 * 8, pools, *state)
        seqs = dev(books.seqs)
        kinds = [forest(r, B, T, V, 1, 0.8) if V < 10000 else None for _ in range(3)]
        if V > 10000:
            tok = torch.randint(0, V, (B, T), **I32)
            par = (torch.arange(T, **I32) - 1).repeat(B, 1).contiguous()
            x = torch.randn((B, T, V), device="cuda").bfloat16()
        else:
            x, tok, par = (dev(a) if isinstance(a, np.ndarray) else a.cuda() for a in kinds[0])
        keep_acc, keep_path = (dev(a) for a in paths(r, n, T, depth))
        acc, path, out = (torch.full(s, -7, **I32) for s in ((B,), (B, depth + 1), (B, depth + 1)))
        status = torch.full((n,), -7, **I32)

        def both(stream):
            sv.specverify_run_greedy_tree(ctx, stream, 1, B, T, V, depth, x, tok, par, None, acc, path, out)
            sv.specverify_cache_keep_path(cache, stream, n, depth + 1, seqs, keep_acc, keep_path, status)

        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        both(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            both(side)
        for i in range(4):
            if V > 10000:
                x.copy_(torch.randn_like(x))
                best = tok.roll(-1, 1).long()[:, :, None]
                x.scatter_(2, best, (torch.rand((B, T, 1), device="cuda") < 0.7).to(x.dtype) * 9)
            else:
                for to, a in zip((x, tok, par), kinds[i % 3]):
                    to.copy_(dev(a) if isinstance(a, np.ndarray) else a.cuda())
            a, p = paths(r, n, T, depth)
            keep_acc.copy_(dev(a))
            keep_path.copy_(dev(p))
            before = [q.clone() for q in pools]
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            got = [q.clone() for q in (acc, path, out, status, *pools)]
            for q, b in zip(pools, before):
                q.copy_(b)
            for q in (acc, path, out, status):
                q.fill_(-7)
            both(None)
            torch.cuda.synchronize()
            for g, q in zip(got, (acc, path, out, status, *pools)):
                assert torch.equal(g, q)
            assert torch.all(status == 0) and acc.max() > 0
        sv.specverify_cache_destroy(cache)
        sv.specverify_destroy(ctx)
