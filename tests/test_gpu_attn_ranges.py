"""Attention over a paged cache at the ends of its ranges: scores so large that one token takes all, windows
and many entries in every form for many rows, sequences of a quarter of a million tokens.  Bounds are those of
test_gpu_attn where nothing else is said."""
import numpy as np
import pytest
import torch

import attn_model as model
from rejection_sampling_verification_row_amd import binding as sv
from test_gpu_attn import E, HALF, TD, Setup

pytestmark = pytest.mark.gpu

# query heads of a key head, nodes and head sizes: one of each form for more than 16 rows
WIDE = [(64, 4, 8), (64, 8, 8), (64, 16, 8), (64, 8, 32), (128, 4, 8), (128, 8, 8), (128, 16, 8), (128, 8, 32),
        (256, 8, 8), (256, 16, 8)]


def scores(s, scale):
    """For each row and head its tokens' places in the pool and their scores, from the definition."""
    st, out = s.step(), {}
    kp = s.pools[0][1].reshape(-1, s.Hk, s.D)
    for i in range(s.n):
        q, a, m, ln, par = st.entry(i)
        for t in range(m):
            at = [st.slot(q, j) for j in [*range(ln), *(ln + b for b in model.sees(par, t))]]
            for h in range(s.H):
                out[a + t, h] = at, scale * (kp[at, h // (s.H // s.Hk)] @ s.q64[a + t, h])
    return out


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,group,m", [(64, 2, 7), (128, 4, 3), (256, 1, 9), (64, 4, 8), (128, 8, 8), (128, 8, 32), (256, 8, 8)])
@pytest.mark.parametrize("scale", [40.0, -40.0])
def test_one_token_takes_all(dt, D, group, m, scale):
    """Where one score leads by more than 40, the other weights are below n e^-40, and the result is
    that token's value: its weight, the same in sum and product but for half a step of bfloat16, and
    two roundings.  The log-sum-exp is that score: D + 6 roundings of sum |q k| and four of itself."""
    s = Setup(dt, 2 * group, 2, D, 8, [70, 9, 300], [m, min(m, 5), m], seed=D + m).device()
    got, lse, status = s.attend(scale)
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    vp = s.pools[1][1].reshape(-1, 2, D)
    S = abs(scale) * np.abs(s.q64).sum(2).max() * np.abs(s.pools[0][1]).max()
    clear = 0
    for (row, h), (at, x) in scores(s, scale).items():
        first, second = np.argsort(x)[::-1][:2]
        if x[first] - x[second] < 40 + 2 * (D + 6) * S * E:
            continue
        clear += 1
        v = vp[at[first], h // group]
        tol = ((HALF["bf16"] if dt == "bf16" else 0) + HALF[dt] * 1.01 + 8 * E) * np.abs(v) + 1e-14
        assert np.all(np.abs(got[row, h] - v) <= tol)
        assert abs(lse[row, h] - x[first]) <= (D + 6) * S * E + 4 * E * abs(x[first])
    assert status.tolist() == [0, 0, 0] and clear >= (2 * m + min(m, 5)) * 2 * group // 2


@pytest.mark.parametrize("D,group,m", WIDE)
@pytest.mark.parametrize("window", [1, 3, 100, 190, 449])
def test_windows_in_every_form_for_many_rows(D, group, m, window):
    """Windows that begin in the nodes, and inside blocks and stages of the cached tokens."""
    s = Setup("bf16", 2 * group, 2, D, 16, [700, 0, 129], [m, m, max(m - 1, 1)], seed=window)
    s.device().check_attend(window=window)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,group,m", [(64, 4, 8), (128, 8, 8), (256, 16, 5)])
def test_many_entries_of_many_rows(dt, D, group, m):
    """More entries than a workgroup has threads, twice over, some of them empty or refused."""
    r = np.random.RandomState(D)
    n = 1100
    s = Setup(dt, group, 1, D, 4, r.randint(0, 25, n).tolist(), r.randint(0, m + 1, n).tolist(), seed=3, max_count=m)
    s.given["counts"][700] = m + 1
    s.given["parents"][s.given["starts"][1050] + 1] = 7 if s.given["counts"][1050] > 1 else -5
    s.device().check_attend()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,group,m,window", [(64, 4, 1, 0), (128, 4, 2, 0), (64, 6, 3, 0), (128, 20, 1, 0), (256, 17, 1, 0),
                                              (128, 6, 3, 200000)])
def test_a_quarter_of_a_million_tokens(dt, D, group, m, window):
    """Tokens all along the sequence, the first and the last among them, hold about half of the weight
    together, so that none of the parts can be missing.  A term of a sum passes at most n / 256 roundings
    in its workgroup, which has no more tokens, and 600 in the joining of at most 768 parts, of which a
    group of lanes adds a quarter or less."""
    ln, scale = 250001, D ** -0.5
    s = Setup(dt, group, 1, D, 64, [ln], [m], seed=D, parents=False)
    st = s.step()
    q, a = st.entry(0)[0], st.entry(0)[1]
    # one query for all heads and nodes, but for a little; keys that score log(n / 24) or so with it
    r = np.random.RandomState(1)
    u = r.standard_normal(D)
    s.q = torch.from_numpy((u + 0.05 * r.standard_normal(s.q64.shape)).astype(np.float32)).to(TD[dt])
    s.q64[:] = s.q.double().numpy()
    places = [0, 1, 31, 32, 63, 64, 65535, 65536, 99999, 131071, 131072, 180000, 200001, 230017, ln - 33, ln - 32, ln - 2, ln - 1]
    t, f = s.pools[0]
    flat, flat64 = t.view(-1, 1, D), f.reshape(-1, 1, D)
    for j in places:
        at = st.slot(q, j)
        flat[at] = torch.from_numpy(u * (np.log(ln / 24.0) + 0.5) / scale / (u @ u)).to(TD[dt])
        flat64[at] = flat[at].double().numpy()
    got, lse, status = s.device().attend(scale, window)
    kp, vp = (p[1].reshape(-1, 1, D) for p in s.pools)
    rows = np.arange(a, a + m)
    want, want_lse, _, _, size = model.attend(st, kp, vp, s.q64, scale, window, 1)
    S = scale * np.abs(s.q64).sum(2).max() * np.abs(kp).max()
    rel = (2 * (D + 6) * S + 16 + ln / 256 + 600) * E
    tol = (rel + (HALF["bf16"] if dt == "bf16" else 0)) * size + HALF[dt] * np.abs(want) * 1.01
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    assert status.tolist() == [0]
    # what one of the places weighs is far above the bounds
    assert np.abs(want[rows]).mean() > 6 * tol[rows].mean()
    assert np.all(np.abs(got - want)[rows] <= tol[rows])
    assert np.all(np.abs(lse - want_lse)[rows] <= rel + 4 * E * np.abs(want_lse[rows]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,group,m", [(64, 2, 7), (128, 4, 3), (256, 1, 9), (64, 4, 8), (128, 8, 8), (128, 8, 32), (256, 8, 8)])
def test_scores_at_the_ends_of_the_range(dt, D, group, m):
    """Keys with the type's lowest value, whose scores of -3.4e38 pass fp32 times log2 e: they have no
    weight, also where they come first, and a row of nothing else is a mean.  A token whose score is as far
    above 0 takes all.  Log-sum-exps as large are off by six roundings, and may round to infinity."""
    s = Setup(dt, 2 * group, 2, D, 8, [300, 40, 90], [m, min(m, 4), m], seed=D + m)
    st, top = s.step(), torch.finfo(TD[dt]).max
    s.q[:, :, 0] = 1.0
    s.q64[:, :, 0] = 1.0
    t, f = s.pools[0]
    flat, flat64 = t.view(-1, 2, D), f.reshape(-1, 2, D)
    places = [(0, j) for j in range(150)] + [(1, j) for j in range(40 + min(m, 4))]
    last = st.entry(2)[2] - 1                        # a leaf
    for i, j in places + [(2, 90 + last)]:
        at = st.slot(st.entry(i)[0], j)
        flat[at, :, 0] = top if i == 2 else -top
        flat64[at, :, 0] = float(top if i == 2 else -top)
    got, lse, status = s.device().attend(1.0)
    kp, vp = (p[1].reshape(-1, 2, D) for p in s.pools)
    with np.errstate(over="ignore"):
        want, want_lse, _, _, size = model.attend(st, kp, vp, s.q64, 1.0, 0, 2)
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    S = np.abs(s.q64).sum(2).max() * np.abs(kp[np.abs(kp) < 1e30]).max()
    rel = (2 * (D + 6) * S + 16 + 400) * E
    tol = (rel + (HALF["bf16"] if dt == "bf16" else 0)) * size + HALF[dt] * np.abs(want) * 1.01
    a0, a1, a2 = (st.entry(i)[1] for i in range(3))
    assert status.tolist() == [0, 0, 0]
    rows = [a + x for a, c in ((a0, m), (a1, min(m, 4)), (a2, m)) for x in range(c)]
    assert np.all(np.abs(got - want)[rows] <= tol[rows])
    a, b = lse[rows], want_lse[rows]
    past = np.isinf(a) & (np.sign(a) == np.sign(b)) & (np.abs(b) * (1 + 6 * E) > np.finfo(np.float32).max)
    assert np.abs(want_lse[a1]).min() > 3e38 and np.abs(want_lse[a2 + last]).min() > 3e38
    with np.errstate(invalid="ignore"):
        assert np.all(past | (np.abs(a - b) <= rel + 6 * E * np.abs(b)))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("group,m", [(2, 6), (2, 30), (8, 33)])
def test_the_last_places_that_a_cache_can_have(dt, group, m):
    """A sequence up to place 2^31 - 3, of which a window is seen: blocks of 32 tokens end at 2^31.  What
    siblings do not see there is NaN."""
    pt, blocks, D = 2718, 790097, 8                  # 2^31 - 2 tokens
    s = Setup(dt, group, 1, D, pt, [0], [m], seed=m)
    q = s.given["seqs"][0]
    s.mb = blocks
    tables = np.full((len(s.blocks), blocks), -1, np.int32)
    tables[q] = 0
    # the places of the nodes and of the window have a page of their own
    tables[q, -1] = s.tables[q, 0]
    tables[q, :-1] = (s.tables[q, 0] + 1) % s.P
    s.tables, s.blocks[q], s.lengths[q] = tables, blocks, pt * blocks - m
    st = s.step()
    ln, a = pt * blocks - m, s.given["starts"][0]
    par = s.given["parents"]
    par[a + m - 2] = par[a + m - 1] = 0              # two leaves
    for x in (m - 2, m - 1):
        at = st.slot(q, ln + x)
        for t, f in s.pools:
            f.reshape(-1, 1, D)[at] = np.nan
            t.view(-1, 1, D)[at] = float("nan")
    window = 50
    got, lse, status = s.device().attend(0.3, window)
    kp, vp = (p[1].reshape(-1, 1, D) for p in s.pools)
    want, want_lse, _, rows, size = model.attend(st, kp, vp, s.q64, 0.3, window, 1)
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    assert status.tolist() == [0]
    clean = [r for r in rows if r < a + m - 2]
    assert np.isnan(got[a + m - 2:a + m]).all() and not np.isnan(want[clean]).any()
    S = 0.3 * np.abs(s.q64).sum(2).max() * np.nanmax(np.abs(kp))
    rel = (2 * (D + 6) * S + 16 + window + m) * E
    tol = (rel + (HALF["bf16"] if dt == "bf16" else 0)) * size + HALF[dt] * np.abs(want) * 1.01
    assert np.all(np.abs(got - want)[clean] <= tol[clean])
    assert np.all(np.abs(lse - want_lse)[clean] <= rel + 4 * E * np.abs(want_lse[clean]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,group,m", [(64, 2, 7), (128, 8, 8)])
def test_scale_zero_takes_the_mean_whatever_the_queries(dt, D, group, m):
    s = Setup(dt, 2 * group, 2, D, 8, [300, 9], [m, 3], seed=D)
    s.q[::2] = float("inf")
    s.q[1::3] = float("nan")
    s.q64[:] = 0.0
    s.device().check_attend(scale=0.0)


@pytest.mark.parametrize("D,group,m", WIDE)
def test_values_near_the_types_largest(D, group, m):
    """A token of a large weight, not among the first, whose values are 1e38: no weight is above 1, so that
    the sums pass fp32 only where the weighted values do."""
    s = Setup("bf16", group, 1, D, 16, [900, 1300], [m, m], seed=D + m, parents=False)
    st, scale = s.step(), D ** -0.5
    r = np.random.RandomState(3)
    u = r.standard_normal(D)
    s.q = torch.from_numpy((u + 0.02 * r.standard_normal(s.q64.shape)).astype(np.float32)).bfloat16()
    s.q64[:] = s.q.double().numpy()
    (kt, kf), (vt, vf) = s.pools
    kt.mul_(0.25)
    kf[:] = kt.double().numpy()
    for i, j in ((0, 500), (1, 777)):
        at = st.slot(st.entry(i)[0], j)
        kt.view(-1, 1, D)[at] = torch.from_numpy(u * 4.5 / scale / (u @ u)).bfloat16()
        kf.reshape(-1, 1, D)[at] = kt.view(-1, 1, D)[at].double().numpy()
        vt.view(-1, 1, D)[at] *= 1e38 / vt.view(-1, 1, D)[at].abs().max()
        vf.reshape(-1, 1, D)[at] = vt.view(-1, 1, D)[at].double().numpy()
    got = s.device().check_attend(scale)
    assert np.isfinite(got).all() and np.abs(got).max() > 1e35


def test_one_pool_for_keys_and_values():
    """An append into it is refused and writes nothing; attention may read both from it."""
    s = Setup("bf16", 4, 2, 64, 8, [30, 20], [5, 4], seed=1).device()
    lib = sv.load()
    status = torch.full((2,), -7, dtype=torch.int32, device="cuda")
    for pool in (0, 1):
        assert lib.specverify_attn_append(s.h, None, pool, pool, 2, 5, s.rows, sv.ctypes.byref(s.nodes), None, s.dk.data_ptr(),
                                          s.wide, s.dv.data_ptr(), s.wide, None, 0, None, 0,
                                          status.data_ptr()) == sv.SPECVERIFY_EINVAL
    out = torch.zeros(s.rows, 4, 64, dtype=torch.bfloat16, device="cuda")
    sv.specverify_attn_attend(s.h, None, 1, 1, 2, 5, s.rows, s.nodes, 0.1, 0, s.dq, s.wide, out, 256)
    torch.cuda.synchronize()
    assert status.tolist() == [-7, -7]
    for (t, _), d in zip(s.pools, s.dpools):
        assert torch.equal(t, d.cpu())
    vp = s.pools[1][1].reshape(-1, 2, 64)
    want, _, _, rows, size = model.attend(s.step(), vp, vp, s.q64, 0.1, 0, 2)
    assert np.all(np.abs(out.double().cpu().numpy() - want)[rows] <= (2.0 ** -7 * size + 1e-4)[rows])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,group,m", [(64, 2, 7), (128, 8, 8)])
def test_the_largest_scale(dt, D, group, m):
    """Scores of 0 at a scale of 2e38: a mean.  Above it the scale's powers of two pass fp32, and the call is
    refused."""
    s = Setup(dt, 2 * group, 2, D, 8, [300, 9], [m, 3], seed=D)
    s.q.zero_()
    s.q64[:] = 0.0
    s.device().check_attend(scale=float(np.float32(2e38)))
    out = torch.full((s.rows, s.H, D), 7.0, dtype=TD[dt], device="cuda")
    for scale in (2.1e38, -2.1e38, 3.4e38):
        with pytest.raises(sv.SpecVerifyError) as e:
            sv.specverify_attn_attend(s.h, None, 0, 1, s.n, s.max_count, s.rows, s.nodes, scale, 0, s.dq, s.wide, out,
                                      s.H * D)
        assert e.value.status == sv.SPECVERIFY_EINVAL
    torch.cuda.synchronize()
    assert torch.all(out == 7)
