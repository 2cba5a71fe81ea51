"""The greedy verify of drafted trees, the move of accepted paths, and a step of tree drafting with all
its calls, against models: ids, paths and moved bytes are equal."""
import numpy as np
import pytest
import torch

import attn_model as model
from gpu_support import dev
from rejection_sampling_verification_row_amd import binding as sv

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def tree(r, m):
    return [-1] + [int(r.randint(0, t)) if r.rand() < 0.6 else t - 1 for t in range(1, m)]


def forest(r, B, T, V, dtype, accept, few=0):
    """Logits whose best id is a child's with probability accept; few: that many distinct values."""
    par = np.array([tree(r, T) for _ in range(B)], np.int32)
    tok = r.randint(0, V, (B, T)).astype(np.int32)
    x = r.standard_normal((B, T, V)).astype(np.float32)
    if few:
        x = np.floor(x * few / 4)
    for b in range(B):
        for i in range(T):
            kids = [c for c in range(T) if c and par[b, c] == i]
            if kids and r.rand() < accept:
                x[b, i, tok[b, r.choice(kids)]] = 9
    x = torch.from_numpy(x).to(torch.bfloat16 if dtype else torch.float32)
    return x, tok, par


def check(ctx, dtype, B, T, V, depth, x, tok, par, counts, misalign=0):
    flat = torch.zeros(x.numel() + misalign, dtype=x.dtype, device="cuda")
    flat[misalign:] = x.reshape(-1).cuda()
    acc, path, out = (torch.full(s, -7, **I32) for s in ((B,), (B, depth + 1), (B, depth + 1)))
    sv.specverify_run_greedy_tree(ctx, None, dtype, B, T, V, depth, flat[misalign:], dev(tok), dev(par),
                                  None if counts is None else dev(counts), acc, path, out)
    torch.cuda.synchronize()
    v = x.double().numpy()
    best = v.argmax(2)                   # numpy takes the first of equals
    for b in range(B):
        want = model.walk(best[b], tok[b], par[b], T if counts is None else int(counts[b]), T, V, depth)
        assert (acc[b].item(), path[b].tolist(), out[b].tolist()) == want, b
    return acc, path, out


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("B,T,V,depth", [(1, 1, 1, 0), (3, 2, 50, 1), (2, 64, 1001, 63), (5, 33, 9000, 6), (40, 16, 33000, 5),
                                         (130, 8, 257, 7), (9, 64, 20000, 3)])
@pytest.mark.parametrize("misalign", [0, 1])
def test_tree_verify(dtype, B, T, V, depth, misalign):
    r = np.random.RandomState(T + V)
    x, tok, par = forest(r, B, T, V, dtype, 0.85)
    counts = None if B % 2 else r.randint(1, T + 1, B).astype(np.int32)
    ctx = sv.specverify_create(0, B, T - 1, V)
    acc, _, _ = check(ctx, dtype, B, T, V, depth, x, tok, par, counts, misalign)
    assert depth == 0 or B < 5 or acc.max().item() > 1
    sv.specverify_destroy(ctx)


@pytest.mark.parametrize("dtype", [0, 1])
def test_ties_go_to_the_lowest_id_and_child(dtype):
    """Rows of few values, siblings with the same token, logits of -inf."""
    r = np.random.RandomState(3)
    x, tok, par = forest(r, 30, 20, 400, dtype, 0.5, few=4)
    tok[:, 5:] = tok[:, 5:6]
    x[:10, :, 7] = 30
    tok[:10, 3:9] = 7
    x[20:, :, 100:] = float("-inf")
    ctx = sv.specverify_create(0, 30, 19, 400)
    check(ctx, dtype, 30, 20, 400, 19, x, tok, par, None)
    sv.specverify_destroy(ctx)


def test_bad_trees_are_refused_alone():
    r = np.random.RandomState(4)
    x, tok, par = forest(r, 9, 12, 300, 1, 0.9)
    counts = np.full(9, 12, np.int32)
    tok[0, 11], tok[1, 1], par[2, 4], par[3, 4] = 300, -1, 4, -1
    counts[4], counts[5], counts[6] = 0, 13, 4
    tok[6, 4:], par[6, 4:] = -9, 99               # behind the count
    tok[7, 0], par[7, 0] = -1, 55                 # node 0's are not read
    ctx = sv.specverify_create(0, 9, 11, 300)
    acc, _, _ = check(ctx, 1, 9, 12, 300, 11, x, tok, par, counts)
    assert [v < 0 for v in acc.tolist()] == [True] * 6 + [False] * 3
    sv.specverify_destroy(ctx)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("B,K,V", [(20, 5, 3001), (256, 8, 20011)])
def test_a_chain_is_the_greedy_verify(dtype, B, K, V):
    r = np.random.RandomState(K)
    T = K + 1
    x = torch.from_numpy(r.standard_normal((B, T, V)).astype(np.float32)).to(torch.bfloat16 if dtype else torch.float32)
    tok = r.randint(0, V, (B, T)).astype(np.int32)
    best = x.double().numpy().argmax(2)
    tok[:, 1:] = np.where(r.rand(B, K) < 0.8, best[:, :K], tok[:, 1:])
    par = np.tile(np.arange(-1, K, dtype=np.int32), (B, 1))
    ctx = sv.specverify_create(0, B, K, V)
    acc, path, out = check(ctx, dtype, B, T, V, K, x, tok, par, None)
    acc2, out2 = torch.empty(B, **I32), torch.empty(B, T, **I32)
    sv.specverify_run_greedy(ctx, None, dtype, B, K, V, x.cuda(), dev(tok[:, 1:]), acc2, out2)
    torch.cuda.synchronize()
    assert torch.equal(acc, acc2) and torch.equal(out, out2)
    sv.specverify_destroy(ctx)


# ---------------------------------------------------------------------------------- paths

class Books:
    def __init__(self, pt, lens, room, token, pools, seed=0):
        r = self.r = np.random.RandomState(seed)
        n = len(lens)
        need = [-(-(ln + m) // pt) for ln, m in zip(lens, room)]
        self.pt, self.P, self.S, self.mb = pt, sum(need) + 2, n + 1, max(need) + 1
        pages = r.permutation(self.P)
        self.seqs = r.permutation(self.S)[:n].astype(np.int32)
        self.tables = np.full((self.S, self.mb), -1, np.int32)
        self.blocks, self.lengths = np.zeros(self.S, np.int32), np.zeros(self.S, np.int32)
        self.refs = np.zeros(self.P, np.int32)
        at = 0
        for s, ln, b in zip(self.seqs, lens, need):
            self.tables[s, :b] = pages[at:at + b]
            self.refs[pages[at:at + b]] = 1
            self.blocks[s], self.lengths[s] = b, ln
            at += b
        self.pools = [r.randint(0, 256, (self.P * pt, token)).astype(np.uint8) for _ in range(pools)]

    def run(self, n, max_count, seqs, accepted, path):
        state = [dev(a) for a in (self.refs, self.tables, self.blocks, self.lengths)]
        pools = [dev(p) for p in self.pools]
        token = self.pools[0].shape[1] if self.pools else 16
        h = sv.specverify_cache_create(0, self.P, self.pt, self.S, self.mb, token * self.pt, pools, *state)
        status = torch.full((n,), -7, **I32)
        sv.specverify_cache_keep_path(h, None, n, max_count, None if seqs is None else dev(seqs), dev(accepted),
                                      dev(path), status)
        torch.cuda.synchronize()
        want = model.keep_path(self.pt, self.P, self.tables, self.blocks, self.lengths, self.pools, n, max_count,
                               seqs, accepted, path)
        assert status.tolist() == want
        for p, q in zip(pools, self.pools):
            assert np.array_equal(p.cpu().numpy(), q)
        for s, a in zip(state, (self.refs, self.tables, self.blocks, self.lengths)):
            assert np.array_equal(s.cpu().numpy(), a)
        sv.specverify_cache_destroy(h)
        return want


def paths(r, n, T, depth):
    acc = r.randint(-1, depth + 1, n).astype(np.int32)
    path = np.full((n, depth + 1), -1, np.int32)
    for i in range(n):
        path[i, :acc[i] + 1] = [0, *sorted(r.permutation(np.arange(1, T))[:acc[i]])][:acc[i] + 1]
    return acc, path


@pytest.mark.parametrize("pt,token,pools,T,depth", [(16, 2048, 4, 64, 63), (1, 16, 1, 8, 7), (4, 12, 3, 9, 4), (8, 6, 2, 20, 10),
                                                    (16, 4112, 2, 33, 8), (5, 48, 7, 64, 20), (16, 16, 0, 8, 4)])
def test_paths_that_overlap_their_destinations(pt, token, pools, T, depth):
    r = np.random.RandomState(T)
    lens = list(r.randint(0, 40, 20))
    b = Books(pt, lens, [T] * 20, token, pools, seed=T)
    acc, path = paths(r, 20, T, depth)
    assert b.run(20, depth + 1, b.seqs, acc, path) == [0] * 20


def test_keep_path_refusals_and_lost_pages():
    b = Books(8, [10, 5, 0, 7, 30, 9, 2, 1, 6], [12] * 9, 32, 2)
    acc = np.array([3, 3, 3, 4, -2, 3, 2, 3, 3], np.int32)
    path = np.tile(np.array([0, 2, 5, 9], np.int32), (9, 1))
    path[0] = [1, 2, 5, 9]
    path[1] = [0, 5, 5, 9]
    path[2] = [0, 2, 5, 90]
    b.blocks[b.seqs[5]] = 1                       # fewer pages than tokens
    path[6, 3] = -4                               # past the accepted ones: not read
    b.seqs[7] = b.seqs[6]                         # named before
    b.tables[b.seqs[8], 1] = -1                   # places 8 .. 15
    assert b.run(9, 4, b.seqs, acc, path) == [-1, -1, -1, -1, -1, -1, 0, -1, 0]
    b = Books(8, [10, 5], [12] * 2, 32, 2)
    b.seqs = np.array([-1, b.S], np.int32)
    assert b.run(2, 4, b.seqs, acc[:2], path[:2]) == [-1, -1]


# ---------------------------------------------------------------------------------- all together

@pytest.mark.parametrize("dt", [0, 1])
def test_steps_of_tree_drafting(dt):
    """Prompts appended and committed, then steps: reserve, append, attend, verify, keep the path,
    commit.  The cache then holds exactly the tokens that were fed on accepted paths, and attention
    over it equals attention over those tokens in a row."""
    r = np.random.RandomState(dt)
    n, H, Hk, D, pt, T, V, depth, layers = 5, 4, 2, 64, 8, 12, 500, 4, 2
    td = torch.bfloat16 if dt else torch.float32
    P, mb, es = 200, 30, 2 if dt else 4
    refs, blocks, lengths = (torch.zeros(k, **I32) for k in (P, n, n))
    tables = torch.full((n, mb), -1, **I32)
    pools = [torch.full((P, pt, Hk, D), float("nan"), dtype=td, device="cuda") for _ in range(2 * layers)]
    cache = sv.specverify_cache_create(0, P, pt, n, mb, pt * Hk * D * es, pools, refs, tables, blocks, lengths)
    attn = sv.specverify_attn_create(cache, dt, H, Hk, D, n, T)
    ctx = sv.specverify_create(0, n, T - 1, V)
    freq = dev((1000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32))
    rot = sv.SpecVerifyRotation(freq, D)
    rand = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).to(td).cuda()  # noqa: E731
    kept = [[[] for _ in range(layers)] for _ in range(n)]        # (key, value) rows as written

    def rows_of(layer):
        at = []
        for s in range(n):
            ln, row = lengths[s].item(), tables[s].tolist()
            at.append([row[j // pt] * pt + j % pt for j in range(ln)])
        return at

    prompts = [9, 1, 20, 8, 16]
    counts, most = dev(np.array(prompts, np.int32)), max(prompts)
    starts = dev(np.cumsum([0, *prompts[:-1]]).astype(np.int32))
    nodes = sv.SpecVerifyNodes(starts=starts, counts=counts)
    sv.specverify_cache_reserve(cache, None, n, None, counts)
    for layer in range(layers):
        k, v = rand(sum(prompts), Hk, D), rand(sum(prompts), Hk, D)
        sv.specverify_attn_append(attn, None, 2 * layer, 2 * layer + 1, n, most, sum(prompts), nodes, rot, k,
                                  Hk * D, v, Hk * D)
        for s in range(n):
            a = int(starts[s])
            kept[s][layer] += [v[a + t].cpu() for t in range(prompts[s])]
    sv.specverify_cache_commit(cache, None, n, None, counts - 1)
    for step in range(6):
        par = torch.tensor([tree(r, T) for _ in range(n)], **I32)
        tok = torch.from_numpy(r.randint(0, V, (n, T)).astype(np.int32)).cuda()
        sizes = dev(r.randint(T // 2, T + 1, n).astype(np.int32))
        status = torch.full((5, n), -7, **I32)
        sv.specverify_cache_reserve(cache, None, n, None, sizes, status[0])
        fed = []
        for layer in range(layers):
            q, k, v = rand(n * T, H, D), rand(n * T, Hk, D), rand(n * T, Hk, D)
            nodes = sv.SpecVerifyNodes(counts=sizes, parents=par.view(-1))
            out = torch.zeros(n * T, H, D, dtype=td, device="cuda")
            lse = torch.zeros(n * T, H, device="cuda")
            sv.specverify_attn_append(attn, None, 2 * layer, 2 * layer + 1, n, T, n * T, nodes, rot, k, Hk * D,
                                      v, Hk * D, q, H * D, q, H * D, status[1])
            sv.specverify_attn_attend(attn, None, 2 * layer, 2 * layer + 1, n, T, n * T, nodes, D ** -0.5, 0, q,
                                      H * D, out, H * D, lse, status[2])
            fed.append((q, k, v, out))
        logits = torch.randn(n, T, V, device="cuda").to(td)
        kid = torch.tensor([[next((c for c in range(T) if c and par[s, c] == i), 0) for i in range(T)] for s in
                            range(n)], device="cuda")
        logits.scatter_(2, tok.long().gather(1, kid)[:, :, None], 9.0)
        acc, path, ids = torch.empty(n, **I32), torch.empty(n, depth + 1, **I32), torch.empty(n, depth + 1, **I32)
        sv.specverify_run_greedy_tree(ctx, None, dt, n, T, V, depth, logits, tok, par, sizes, acc, path, ids)
        sv.specverify_cache_keep_path(cache, None, n, depth + 1, None, acc, path, status[3])
        sv.specverify_cache_commit(cache, None, n, None, acc, status[4])
        torch.cuda.synchronize()
        assert torch.all(status == 0) and torch.all(acc >= 0)
        for layer in range(layers):
            for s in range(n):
                kept[s][layer] += [fed[layer][2][s * T + i].cpu() for i in path[s].tolist() if i >= 0]
    assert sum(len(kept[s][0]) for s in range(n)) > sum(prompts) + 6 * n
    for layer in range(layers):
        kp, vp = (pools[2 * layer + i].double().cpu().numpy().reshape(-1, Hk, D) for i in (0, 1))
        for s, at in enumerate(rows_of(layer)):
            assert len(at) == len(kept[s][layer])
            assert np.array_equal(vp[at], torch.stack(kept[s][layer]).double().numpy())
        # one token more for each sequence, over what is now in the cache
        sv.specverify_cache_reserve(cache, None, n, None, torch.ones(n, **I32))
        q, k, v = rand(n, H, D), rand(n, Hk, D), rand(n, Hk, D)
        out = torch.zeros(n, H, D, dtype=td, device="cuda")
        sv.specverify_attn_append(attn, None, 2 * layer, 2 * layer + 1, n, 1, n, None, rot, k, Hk * D, v, Hk * D)
        sv.specverify_attn_attend(attn, None, 2 * layer, 2 * layer + 1, n, 1, n, None, D ** -0.5, 0, q, H * D,
                                  out, H * D)
        torch.cuda.synchronize()
        kp, vp = (pools[2 * layer + i].double().cpu().numpy().reshape(-1, Hk, D) for i in (0, 1))
        st = model.Step(pt, P, tables.cpu().numpy(), blocks.cpu().numpy(), lengths.cpu().numpy(), n, 1, n)
        want, _, _, _, size = model.attend(st, kp, vp, q.double().cpu().numpy(), D ** -0.5, 0, Hk)
        tol = 2.0 ** -7 if dt else 1e-5
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol * (size + np.abs(want)))
    sv.specverify_destroy(ctx)
    sv.specverify_attn_destroy(attn)
    sv.specverify_cache_destroy(cache)
