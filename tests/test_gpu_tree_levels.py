"""Greedy verify of drafted trees whose rows are read depth by depth, against the definition: batches of
large trees, of which a walk needs few rows.  Ids, paths and lengths are equal."""
import numpy as np
import pytest
import torch

import attn_model as model
from gpu_support import dev
from rejection_sampling_verification_row_amd import binding as sv

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")
TD = {0: torch.float32, 1: torch.bfloat16}


def tree(r, T, far):
    return [-1] + [int(r.randint(0, t)) if r.rand() < far else t - 1 for t in range(1, T)]


def forest(r, B, T, V, dtype, accept, few=0, misalign=0, far=0.3):
    """Logits on the device, from an element `misalign` on; a row's best id is a child's with probability
    accept.  few: that many distinct values, so that maxima are tied."""
    par = np.array([tree(r, T, far) for _ in range(B)], np.int32)
    tok = r.randint(0, V, (B, T)).astype(np.int32)
    g = torch.Generator(device="cuda").manual_seed(int(r.randint(1 << 30)))
    flat = torch.zeros(B * T * V + misalign, dtype=TD[dtype], device="cuda")
    x = flat[misalign:].view(B, T, V)
    for b in range(0, B, 8):
        y = torch.randn(x[b:b + 8].shape, generator=g, device="cuda")
        x[b:b + 8] = (y * few / 4).floor() if few else y
    best = np.full((B, T), -1)
    for b in range(B):
        for i in range(T):
            kids = [c for c in range(i + 1, T) if par[b, c] == i]
            if kids and r.rand() < accept:
                best[b, i] = tok[b, r.choice(kids)]
    at = np.argwhere(best >= 0)
    if len(at):
        b, i = (torch.from_numpy(a).cuda() for a in at.T.copy())
        x[b, i, torch.from_numpy(best[best >= 0]).cuda()] = 9.0
    return x, tok, par


def lowest_best(x):
    """The lowest id among each row's maxima, [B][T]."""
    ids = torch.arange(x.shape[2], device="cuda")
    return np.stack([torch.where(y == y.amax(1, keepdim=True), ids, x.shape[2]).amin(1).cpu().numpy() for y in x])


def check(dtype, x, tok, par, depth, counts=None, calls=1):
    B, T, V = x.shape
    ctx = sv.specverify_create(0, B, T - 1, V)
    best = lowest_best(x)
    want = [model.walk(best[b], tok[b], par[b], T if counts is None else int(counts[b]), T, V, depth) for b in range(B)]
    dtok, dpar, dcounts = dev(tok), dev(par), None if counts is None else dev(counts)
    for _ in range(calls):
        acc, path, out = (torch.full(s, -7, **I32) for s in ((B,), (B, depth + 1), (B, depth + 1)))
        sv.specverify_run_greedy_tree(ctx, None, dtype, B, T, V, depth, x, dtok, dpar, dcounts, acc, path, out)
        torch.cuda.synchronize()
        for b in range(B):
            assert (acc[b].item(), path[b].tolist(), out[b].tolist()) == want[b], b
    sv.specverify_destroy(ctx)
    return [w[0] for w in want]


# trees, nodes, ids, depth: walks that end early and that go all the way down; a row's end inside a
# group of 16 bytes; one chunk of a row's and many
SHAPES = [(96, 64, 32000, 3), (192, 64, 32000, 12), (40, 50, 65537, 5), (256, 33, 9001, 1), (64, 8, 152064, 0),
          (24, 64, 128255, 8)]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("B,T,V,depth", SHAPES)
@pytest.mark.parametrize("misalign", [0, 1])
def test_walks(dtype, B, T, V, depth, misalign):
    r = np.random.RandomState(B + depth)
    x, tok, par = forest(r, B, T, V, dtype, 0.9, misalign=misalign)
    counts = r.randint(1, T + 1, B).astype(np.int32) if misalign else None
    acc = check(dtype, x, tok, par, depth, counts, calls=2)
    assert min(acc) == 0 and max(acc) == depth


@pytest.mark.parametrize("dtype", [0, 1])
def test_ties_go_to_the_lowest_id_and_child(dtype):
    """Rows of few values, siblings with the same token, rows that are -inf but for few ids or altogether."""
    r = np.random.RandomState(11)
    x, tok, par = forest(r, 96, 64, 32000, dtype, 0.6, few=4)
    tok[:, 20:] = tok[:, 20:21]
    x[:24, :, 31999] = 30
    x[:24, :, 8192 * 3] = 30
    tok[:24, 1:30] = 8192 * 3
    x[24:40, :, 100:] = float("-inf")
    x[40:56] = float("-inf")
    tok[40:56, 1:] = 0
    acc = check(dtype, x, tok, par, 3)
    assert max(acc[:24]) == 3 and max(acc[40:56]) == 3


@pytest.mark.parametrize("dtype", [0, 1])
def test_bad_trees_are_refused_alone(dtype):
    r = np.random.RandomState(12)
    B, T, V = 96, 64, 32000
    x, tok, par = forest(r, B, T, V, dtype, 0.9)
    counts = np.full(B, T, np.int32)
    bad = {0: "id", 7: "low id", 8: "parent", 30: "own parent", 31: "count 0", 64: "count above", 95: "negative parent"}
    tok[0, 63], tok[7, 1], par[8, 4], par[30, 9] = V, -1, 5, 9
    counts[31], counts[64], par[95, 63] = 0, T + 1, -1
    counts[50] = 4
    tok[50, 4:], par[50, 4:] = -9, 99             # behind the count
    tok[51, 0], par[51, 0] = -1, 55               # node 0's are not read
    acc = check(dtype, x, tok, par, 3, counts)
    assert [b for b in range(B) if acc[b] < 0] == sorted(bad)


@pytest.mark.parametrize("dtype", [0, 1])
def test_the_start_of_a_chain_is_the_greedy_verify(dtype):
    """A chain's walk over at most `depth` drafts: the greedy verify of its first `depth` ones."""
    r = np.random.RandomState(13)
    B, T, V, depth = 96, 64, 32000, 3
    x, tok, par = forest(r, B, T, V, dtype, 0.8, far=0.0)
    acc = check(dtype, x, tok, par, depth)
    ctx = sv.specverify_create(0, B, depth, V)
    acc2, out2 = torch.empty(B, **I32), torch.empty(B, depth + 1, **I32)
    sv.specverify_run_greedy(ctx, None, dtype, B, depth, V, x[:, :depth + 1].contiguous(),
                             dev(np.ascontiguousarray(tok[:, 1:depth + 1])), acc2, out2)
    ctx3 = sv.specverify_create(0, B, T - 1, V)
    acc3, path3, out3 = (torch.empty(s, **I32) for s in ((B,), (B, depth + 1), (B, depth + 1)))
    sv.specverify_run_greedy_tree(ctx3, None, dtype, B, T, V, depth, x, dev(tok), dev(par), None, acc3, path3, out3)
    torch.cuda.synchronize()
    assert acc2.tolist() == acc and torch.equal(acc2, acc3) and torch.equal(out2, out3)
    sv.specverify_destroy(ctx)
    sv.specverify_destroy(ctx3)


@pytest.mark.parametrize("dtype", [0, 1])
def test_timing_spans_every_depth(dtype):
    """The timed launches of the argmax kind: one for a call, from the first depth's start to the last's
    end.  All walks go down to the end, so that 13 depths, which wait for one another, take several
    times what one does; and all of the call takes longer than they do."""
    r = np.random.RandomState(14)
    B, T, V = 192, 64, 32000
    x, tok, par = forest(r, B, T, V, dtype, 1.0, far=0.0)
    ctx = sv.specverify_create(0, B, T - 1, V)
    us = {}
    for depth in (0, 12):
        acc, path, out = (torch.empty(s, **I32) for s in ((B,), (B, depth + 1), (B, depth + 1)))
        args = (ctx, None, dtype, B, T, V, depth, x, dev(tok), dev(par), None, acc, path, out)
        for _ in range(3):
            sv.specverify_run_greedy_tree(*args)
        sv.specverify_profile_begin(ctx, 8, ["row_argmax", "greedy_emit"])
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for _ in range(8):
            sv.specverify_run_greedy_tree(*args)
        end.record()
        ms = sv.specverify_profile_launches(ctx, "row_argmax")
        emit = sv.specverify_profile_launches(ctx, "greedy_emit")
        sv.specverify_profile_end(ctx)
        assert len(ms) == len(emit) == 8 and min(ms) > 0 and acc.min().item() == depth
        assert sum(ms) + sum(emit) <= begin.elapsed_time(end) * 1.05
        us[depth] = sorted(ms)[4] * 1e3
    assert us[12] >= 4 * us[0], us
    sv.specverify_destroy(ctx)
