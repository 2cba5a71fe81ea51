"""Rows whose large logits stand in one place, cut by top-k and min-p together: most waves meet their
first loads before min-p's bound is known, count them or list everything, and what is passed over
later lies above what was counted.  Compared like test_gpu_filter.py."""
import numpy as np
import pytest

import filter_model as model
from test_gpu_filter import (BF16, F32, PROB_RTOL, as_dtype, check_sample, check_verify, ctx,  # noqa: F401
                             rows, run_sample)

pytestmark = pytest.mark.gpu

LOWEST = -3.3895313892515355e38


def block(r, n, V, low):
    """All `low` but one block of ids, at any place."""
    x = np.full((n, V), low, np.float32)
    for i in range(n):
        size = r.randint(2000, 6000)
        at = r.randint(0, V - size)
        x[i, at:at + size] = rows(r, 1, size, 2.5)[0] * r.uniform(0.7, 1.3)
    return x


def peaks(r, n, V):
    """A block of close logits with a few far above them, the rest masked."""
    x = np.full((n, V), -np.inf, np.float32)
    for i in range(n):
        at = r.randint(0, V - 4000)
        x[i, at:at + 4000] = 20 + r.randn(4000)
        x[i, at + r.randint(0, 4000, 3)] = r.uniform(27, 28, 3)
    return x


def late(r, n, V):
    """The first half of each wave's range at or below zero, most of the rest a little above, one
    peak: few of the first lie at the top of their bin."""
    per = ((V + 3) // 4 + 1023) // 1024 * 256          # ids of a wave's range of float32 groups
    x = -1.0 - 0.2 * r.rand(n, V)
    half = np.arange(V) % per < per // 2
    x[:, ~half] = 1.0 + 0.5 * r.rand(n, (~half).sum())
    for i in range(n):
        first = np.flatnonzero(half)
        x[i, r.choice(first, r.randint(5, 32), replace=False)] = -0.5 - 0.001 * r.rand()
        x[i, r.choice(np.flatnonzero(~half))] = 40.0 + r.rand()
    return x.astype(np.float32)


ROWS = {"block in -inf": lambda r, n, V: block(r, n, V, -np.inf),
        "block in the lowest": lambda r, n, V: block(r, n, V, LOWEST),
        "peaks": peaks, "late": late}


def cuts(r, n, ks):
    return dict(T=r.uniform(0.5, 1.2, n).astype(np.float32), k=r.choice(ks, n).astype(np.int32),
                p=np.ones(n, np.float32), m=r.uniform(0.05, 0.3, n).astype(np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [50257, 128256])
@pytest.mark.parametrize("kind", ROWS)
def test_sample_a_block_of_ids_by_top_k_and_min_p(ctx, kind, V, dtype):
    r = np.random.RandomState(len(kind) + V)
    n = 100
    q = cuts(r, n, [10, 20, 24, 33, 50, 60])
    q["k"][:8] = [300, 1024] * 4
    check_sample(ctx, ROWS[kind](r, n, V), dtype, q, r.rand(n).astype(np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ROWS)
def test_verify_a_block_of_ids_by_top_k_and_min_p(ctx, kind, dtype):
    r = np.random.RandomState(len(kind))
    B, K, V = 12, 2, 128256
    f = cuts(r, B, [10, 20, 24, 50, 300])
    t = ROWS[kind](r, B * (K + 1), V).reshape(B, K + 1, V)
    for b in range(B):                               # one mask for a sequence's rows
        t[b] = t[b, 0]
    t = np.where(t > -256, t + 0.3 * rows(r, B * (K + 1), V, 1).reshape(t.shape), t).astype(np.float32)
    d = np.where(t[:, :K] > -256, t[:, :K] + 0.3 * rows(r, B * K, V, 1).reshape(B, K, V),
                 t[:, :K]).astype(np.float32)
    tb, tv = as_dtype(t, dtype)
    db, dv = as_dtype(d, dtype)
    x = np.zeros((B, K), np.int32)
    for b in range(B):
        for j in range(K):
            q = model.law(dv[b, j], *(f[c][b] for c in "Tkpm"))[0]
            x[b, j] = r.choice(V, p=q / q.sum())
    check_verify(ctx, (tb, tv, db, dv, x, r.rand(B, K + 1).astype(np.float32)), dtype, f, f, same=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("low", [-257.0, -300.0, -700.0])
def test_ids_masked_by_a_value_that_still_weighs_something(ctx, low, dtype):
    """Fewer ids than top-k's above the mask, or above min-p's bound; the masked ones are kept where
    top-k reaches them and min-p does not, and only there."""
    r = np.random.RandomState(int(-low))
    n, V = 48, 50257
    x = np.full((n, V), low, np.float32)
    for i in range(n):
        at = r.choice(V, r.choice([5, 30, 400]), replace=False)
        x[i, at] = rows(r, 1, len(at))[0]
    q = cuts(r, n, [20, 50, 1000, 1025])
    q["m"][:] = r.choice([0.0, 1e-20, 0.1], n)
    q["T"][:] = r.choice([0.7, 1.5, 60.0], n)
    u = r.rand(n).astype(np.float32)
    bits, val = as_dtype(x, dtype)
    tok, prob, mar = model.sample(val, u, q["T"], q["k"], q["p"], q["m"])
    for i in np.flatnonzero(q["m"] == np.float32(1e-20)):
        # the model's gap between a weight and m is absolute: here a relative one says how clear it is
        v = val[i].astype(np.float64)
        gap = np.abs(np.exp((v - v.max()) / float(q["T"][i])) / float(q["m"][i]) - 1).min()
        mar[i] = min(gap, model.draw(model.law(val[i], q["T"][i], int(q["k"][i]), 1.0, q["m"][i])[0], u[i])[1])
    clear = mar > model.CLEAR
    assert clear.mean() > 0.9
    g, gp = run_sample(ctx, bits, dtype, q, u)
    assert np.array_equal(g[clear], tok[clear]), (np.flatnonzero(g != tok), g, tok)
    np.testing.assert_allclose(gp[clear], prob[clear], rtol=PROB_RTOL, atol=2.0 ** -149)
