"""Rows that are hard for a cut by counting: crowded bins, runs of equal values at a cut, orders that
defeat a running bound, parameters at the ends of their ranges.  Compared like test_gpu_filter.py:
ids equal wherever the model's decisions are clear of rounding."""
import numpy as np
import pytest
import torch

import filter_model as model
from gpu_support import dev
from rejection_sampling_verification_row_amd import binding as sv
from test_gpu_filter import (BF16, F32, as_dtype, check_sample, check_verify, ctx, filt,  # noqa: F401
                             params, rows, run_sample, run_verify, workload)

pytestmark = pytest.mark.gpu


def plain(n):
    return dict(T=np.ones(n, np.float32), k=np.zeros(n, np.int32), p=np.ones(n, np.float32),
                m=np.zeros(n, np.float32))


CROWDS = {
    "one bin": lambda r, s: 5.0 + r.uniform(0, 2.0 ** -6, s),
    "one bin, half of it equal": lambda r, s: np.where(r.rand(*s) < 0.5, 5.0 + 2.0 ** -8,
                                                       5.0 + r.uniform(0, 2.0 ** -6, s)),
    "one negative bin": lambda r, s: -5.0 - r.uniform(0, 2.0 ** -6, s),
    "two bins": lambda r, s: 4.0 + r.uniform(-2.0 ** -6, 2.0 ** -6, s),
    "a part of a bin": lambda r, s: 5.0 + r.uniform(0, 2.0 ** -19, s),
    "above the window": lambda r, s: 300.0 + r.uniform(0, 3, s),
    "around zero": lambda r, s: r.uniform(-1e-9, 1e-9, s),
    "below the window": lambda r, s: -300.0 - r.uniform(0, 3, s),
    "a crowd under a peak": lambda r, s: np.where(r.rand(*s) < 2e-3, r.uniform(6, 9, s),
                                                  5.0 + r.uniform(0, 2.0 ** -6, s)),
}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("crowd", CROWDS)
def test_sample_crowded_rows(ctx, crowd, dtype):
    r = np.random.RandomState(len(crowd))
    n, V = 20, 20011
    x = CROWDS[crowd](r, (n, V)).astype(np.float32)
    q, u = plain(n), r.rand(n).astype(np.float32)
    q["k"][:10] = [1, 2, 900, 1023, 1024, 1025, 5000, 15000, V - 1, V]
    q["p"][5:] = r.uniform(0.001, 0.999, 15)
    q["T"][15:] = 0.01
    check_sample(ctx, x, dtype, q, u)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("crowd", ["one bin", "one bin, half of it equal", "above the window",
                                   "a crowd under a peak"])
def test_verify_crowded_rows(ctx, crowd, dtype):
    r = np.random.RandomState(len(crowd) + 1)
    B, K, V = 12, 3, 9001
    t, d = CROWDS[crowd](r, (B, K + 1, V)), CROWDS[crowd](r, (B, K, V))
    f = plain(B)
    f["k"] = np.array([0, 1, 40, 1024, 1500, 4000, 8000, 8999, 9000, 0, 0, 0], np.int32)
    f["p"][6:] = r.uniform(0.1, 0.99, 6)
    d[::2] = t[::2, :K]                              # some positions accept, some reject
    tb, tv = as_dtype(t, dtype)
    db, dv = as_dtype(d, dtype)
    x = np.zeros((B, K), np.int32)
    for b in range(B):
        for j in range(K):
            q = model.law(dv[b, j], *(f[c][b] for c in "Tkpm"))[0]
            x[b, j] = r.choice(V, p=q / q.sum())
    check_verify(ctx, (tb, tv, db, dv, x, r.rand(B, K + 1).astype(np.float32)), dtype, f, f, same=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("order", ["ascending", "descending", "best last", "best first", "saw"])
def test_sample_orders(ctx, order, dtype):
    """Where the large logits stand decides how much of a row a running bound can pass over."""
    r = np.random.RandomState(3)
    n, V = 18, 32003
    x = np.sort(rows(r, n, V), axis=1)
    if order == "descending":
        x = x[:, ::-1]
    elif order != "ascending":
        best, rest = x[:, -300:].copy(), x[:, :-300].copy()
        r.shuffle(rest.T)
        x = np.concatenate([best, rest] if order == "best first" else [rest, best], axis=1)
        if order == "saw":                           # a large one in every group of the loads
            x = np.sort(x, axis=1).reshape(-1)[: n * V].reshape(n, V)[:, np.argsort(np.arange(V) % 7, kind="stable")]
    q = params(r, n, "mixed")
    q["k"][::3] = [1, 50, 1024, 1025, 2000, 31000]
    q["p"][::3], q["m"][::3] = 1.0, 0.0
    check_sample(ctx, np.ascontiguousarray(x), dtype, q, r.rand(n).astype(np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_parameters_at_the_ends(ctx, dtype):
    r = np.random.RandomState(14)
    n, V = 16, 12289
    x = rows(r, n, V)
    _, val = as_dtype(x, dtype)
    q = plain(n)
    q["p"][0], q["p"][1], q["p"][2] = 0.0, 1e-30, np.float32(1) - np.float32(2.0 ** -24)
    q["m"][3], q["m"][4] = 1.0, 1e-38
    q["T"][5], q["T"][6], q["T"][7] = 1e-30, 3e38, 1e-45
    q["k"][8], q["k"][9], q["k"][10] = 1, V - 1, -(1 << 31)
    q["T"][11], q["k"][11] = 0.0, 7
    q["T"][12], q["p"][12], q["m"][12] = 3e38, 0.5, 1.0
    q["p"][13], q["m"][13] = 0.0, 1.0
    q["T"][14], q["p"][14] = 1e-30, 0.3
    u = (r.randint(0, 1 << 20, n) / float(1 << 20)).astype(np.float32)
    tok, prob, mar = model.sample(val, u, q["T"], q["k"], q["p"], q["m"])
    g, gp = run_sample(ctx, as_dtype(x, dtype)[0], dtype, q, u)
    clear = mar > model.CLEAR
    clear[[0, 1, 3, 5, 7, 8, 11, 13, 14]] = True     # nothing but the largest, and its ties
    assert np.array_equal(g[clear], tok[clear])
    top = np.argmax(val, axis=1)
    assert all(g[i] == top[i] and gp[i] == 1 for i in (0, 1, 8, 11, 13))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("low", [-np.inf, -3.3895313892515355e38, -1e9, -257.0])
@pytest.mark.parametrize("T", [0.7, 90.0])
def test_verify_masked_ids(ctx, low, T, dtype):
    """Most ids masked in both models' rows; at T = 90 the low value -257 still weighs something."""
    r = np.random.RandomState(int(T))
    B, K, V = 8, 3, 4003
    ft = params(r, B, "mixed")
    ft["T"][ft["T"] > 0] *= T
    gone = r.rand(B, 1, V) < 0.8
    gone[:, :, 5] = False
    t = rows(r, B * (K + 1), V).reshape(B, K + 1, V)
    d = t[:, :K] + rows(r, B * K, V, 0.5).reshape(B, K, V)
    t, d = np.where(gone, low, t).astype(np.float32), np.where(gone, low, d).astype(np.float32)
    tb, tv = as_dtype(t, dtype)
    db, dv = as_dtype(d, dtype)
    x = np.zeros((B, K), np.int32)
    for b in range(B):
        for j in range(K):
            q = model.law(dv[b, j], *(ft[c][b] for c in "Tkpm"))[0]
            x[b, j] = r.choice(V, p=q / q.sum())
    check_verify(ctx, (tb, tv, db, dv, x, r.rand(B, K + 1).astype(np.float32)), dtype, ft, ft, same=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("k", [40, 300, 1500, 6000, 15000])
def test_min_p_leaves_fewer_than_top_k(ctx, k, dtype):
    """What lies below min-p's bound is not looked at, so that fewer than k ids may be seen."""
    r = np.random.RandomState(k)
    n, V = 24, 20011
    q = plain(n)
    q["k"][:] = k
    q["m"][:] = 10.0 ** r.uniform(-6, -0.5, n)
    q["T"][:] = r.uniform(0.3, 2.5, n)
    check_sample(ctx, rows(r, n, V), dtype, q, r.rand(n).astype(np.float32))
    f = {c: a[:8] for c, a in q.items()}
    check_verify(ctx, workload(r, 8, 2, 5003, dtype, f, f), dtype, f, f, same=True)


@pytest.mark.parametrize("bits", [0x7F800001, 0xFF800001, 0x7FC00000, 0xFFC00000, 0xFFFFFFFF])
@pytest.mark.parametrize("kind", ["", "k", "p", "m"])
def test_a_nan_of_any_sign_anywhere_ends_its_row(ctx, bits, kind):
    """Also in a place that a bound from k or min-p would pass over."""
    r = np.random.RandomState(bits & 0xff)
    n, V = 12, 16001
    q, u = params(r, n, kind), r.rand(n).astype(np.float32)
    if "k" in kind:
        q["k"][:] = 1 + np.arange(n)
    x = rows(r, n, V)
    where = [0, 1, 255, 4095, 8000, 15999, 16000]
    for i, w in enumerate(where):
        x[i].view(np.uint32)[w] = bits
    g, gp = run_sample(ctx, x, F32, q, u)
    assert np.all(g[:7] == -1) and np.all(np.isnan(gp[:7])) and np.all(g[7:] >= 0)
    b = as_dtype(np.where(np.isnan(x), 0, x), BF16)[0].copy()
    for i, w in enumerate(where):
        b[i].view(np.uint16)[w] = (bits >> 16) | (1 if bits & 0x7fffffff == 0x7f800001 else 0)
    g, gp = run_sample(ctx, b, BF16, q, u)
    assert np.all(g[:7] == -1) and np.all(np.isnan(gp[:7])) and np.all(g[7:] >= 0)
    f = params(r, 3, kind)
    acc, out, pr = run_verify(ctx, x[:12].reshape(3, 4, V), np.ascontiguousarray(rows(r, 9, V)).reshape(3, 3, V),
                              F32, f, f, np.zeros((3, 3), np.int32), np.full((3, 4), 0.5, np.float32))
    assert np.all(acc[:2] == -1) and np.all(out[:2] == -1) and acc[2] >= 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("k", [500, 4000, 9000, 20000])
def test_verify_draws_from_few_and_from_many_kept_ids(ctx, k, dtype):
    """A target's kept ids listed, or too many for it; with ties at both rows' cuts, and the draft
    equal to the target but for a few ids, so that the residual is small."""
    r = np.random.RandomState(k)
    B, K, V = 10, 2, 50021
    t = (np.round(rows(r, B * (K + 1), V) * 4) / 4).reshape(B, K + 1, V)
    d = t[:, :K].copy()
    for b in range(B):
        for j in range(K):
            at = r.permutation(V)[:50]
            d[b, j, at] += 1.0
    f = plain(B)
    f["k"][:] = k + np.arange(B)
    f["T"][:] = 1.4426950408889634
    tb, tv = as_dtype(t, dtype)
    db, dv = as_dtype(d, dtype)
    x = np.zeros((B, K), np.int32)
    for b in range(B):                               # half of them where the draft promises too much
        for j in range(K):
            x[b, j] = np.argmax(dv[b, j] - tv[b, j] + 0.01 * dv[b, j]) if b % 2 else np.argmax(tv[b, j])
    check_verify(ctx, (tb, tv, db, dv, x, r.rand(B, K + 1).astype(np.float32)), dtype, f, f, same=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_every_run_gives_the_same_bits(ctx, dtype):
    r = np.random.RandomState(23)
    n, V = 64, 40009
    x, q, u = rows(r, n, V), params(r, n, "mixed"), r.rand(n).astype(np.float32)
    b = as_dtype(x, dtype)[0]
    first = run_sample(ctx, b, dtype, q, u)
    f = params(r, 8, "mixed")
    w = workload(r, 8, 3, 7001, dtype, f, f)
    verified = run_verify(ctx, w[0], w[2], dtype, f, f, w[4], w[5])
    for _ in range(5):
        again = run_sample(ctx, b, dtype, q, u)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])
        for a, c in zip(verified, run_verify(ctx, w[0], w[2], dtype, f, f, w[4], w[5])):
            assert np.array_equal(a, c)


def test_rows_further_apart_than_32_bits(ctx):
    r = np.random.RandomState(25)
    n, V, stride = 2, 5003, (1 << 31) + 9
    x, q, u = rows(r, n, V), params(r, n, "kp"), r.rand(n).astype(np.float32)
    bits, _ = as_dtype(x, BF16)
    want, _ = run_sample(ctx, bits, BF16, q, u)
    wide = torch.zeros(stride + V, dtype=torch.bfloat16, device="cuda")
    for i in range(n):
        wide[i * stride: i * stride + V] = torch.from_numpy(bits[i]).cuda().view(torch.bfloat16)
    tok = torch.zeros(n, dtype=torch.int32, device="cuda")
    sv.specverify_sample_filtered(ctx, None, BF16, n, V, stride, filt(q), wide, dev(u), tok)
    assert np.array_equal(tok.cpu().numpy(), want)


def test_rows_behind_the_last_are_left_as_they_were(ctx):
    r = np.random.RandomState(26)
    n, V = 5, 3001
    x, q, u = rows(r, n, V), params(r, n, "mixed"), r.rand(n).astype(np.float32)
    tok = torch.full((n + 3,), -7, dtype=torch.int32, device="cuda")
    pr = torch.full((n + 3,), -7.0, device="cuda")
    sv.specverify_sample_filtered(ctx, None, F32, n, V, V, filt(q), dev(x), dev(u), tok, pr)
    assert torch.all(tok[n:] == -7) and torch.all(pr[n:] == -7) and torch.all(tok[:n] >= 0)
