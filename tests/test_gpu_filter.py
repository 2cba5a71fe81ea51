"""The cut laws on the GPU against the 64-bit model: tokens and lengths equal wherever the model's
decisions are clear of rounding (which the inputs here are made to be), probabilities to the
rounding of their float32 output: half a step, 2^-24 relative, plus what the fp64 sums carry."""
import numpy as np
import pytest
import torch

import filter_model as model
from gpu_support import dev, dev_offset
from rejection_sampling_verification_row_amd import binding as sv

pytestmark = pytest.mark.gpu

F32, BF16 = sv.SPECVERIFY_F32, sv.SPECVERIFY_BF16
PROB_RTOL = 2.0 ** -24 * 1.01
NAMES = dict(T="temperature", k="top_k", p="top_p", m="min_p")


@pytest.fixture(scope="module")
def ctx():
    h = sv.specverify_create(0, 512, 63, sv.SPECVERIFY_MAX_VOCAB)
    yield h
    sv.specverify_destroy(h)


def bf16_bits(x):
    """float32 -> bfloat16 patterns, nearest even; the values they stand for."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)
    return t.view(torch.int16).numpy(), t.float().numpy()


def as_dtype(x, dtype):
    """(device bytes as numpy, values as float32) of logits x."""
    x = np.ascontiguousarray(x, np.float32)
    return (x, x) if dtype == F32 else bf16_bits(x)


def params(r, n, kind):
    """n rows' parameters; "mixed" has every sort of request, greedy among them."""
    q = dict(T=r.uniform(0.3, 1.5, n), k=r.randint(1, 80, n), p=r.uniform(0.3, 0.999, n),
             m=r.uniform(0.01, 0.3, n))
    on = r.rand(4, n)
    if kind == "mixed":
        q["T"] = np.where(on[0] < 0.15, 0.0, q["T"])
        q["k"] = np.where(on[1] < 0.5, r.choice([0, -3, 1 << 30], n), q["k"])
        q["p"] = np.where(on[2] < 0.4, 1.0, q["p"])
        q["m"] = np.where(on[3] < 0.5, 0.0, q["m"])
    else:
        q = {c: (q[c] if c in kind else dict(T=np.ones(n), k=np.zeros(n, int), p=np.ones(n),
                                             m=np.zeros(n))[c]) for c in q}
    return {c: q[c].astype(np.int32 if c == "k" else np.float32) for c in q}


def filt(q):
    return sv.SpecVerifyFilter(**{NAMES[c]: dev(q[c]) for c in q})


def run_sample(ctx, x, dtype, q, u, stride=None, misalign=0, probs=True, stream=None):
    n, V = x.shape
    if stride:
        wide = np.zeros((n, stride), x.dtype)
        wide[:, :V] = x
        x = wide
    d = dev_offset(x, misalign) if misalign else dev(x)
    tok = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    pr = torch.full((n,), -7.0, device="cuda") if probs else None
    sv.specverify_sample_filtered(ctx, stream, dtype, n, V, stride or V, filt(q), d, dev(u), tok, pr)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), None if pr is None else pr.cpu().numpy()


def check_sample(ctx, x, dtype, q, u, **kw):
    bits, val = as_dtype(x, dtype)
    tok, prob, mar = model.sample(val, u, q["T"], q["k"], q["p"], q["m"])
    clear = mar > model.CLEAR
    assert clear.mean() > 0.9
    g, gp = run_sample(ctx, bits, dtype, q, u, **kw)
    assert np.array_equal(g[clear], tok[clear]), (np.flatnonzero(g != tok), g, tok)
    assert np.all((g >= 0) == (tok >= 0)) and np.all(g < x.shape[1])
    if gp is not None:
        np.testing.assert_allclose(gp[clear], prob[clear], rtol=PROB_RTOL, atol=2.0 ** -149)


def rows(r, n, V, scale=3.0):
    return (r.standard_normal((n, V)) * scale).astype(np.float32)


SIZES = [1, 2, 3, 7, 8, 63, 64, 65, 511, 1000, 1023, 1024, 1025, 4095, 8191, 8192, 8193, 16385,
         32000, 50257]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", SIZES)
def test_sample_sizes(ctx, V, dtype):
    r = np.random.RandomState(V)
    n = 12
    check_sample(ctx, rows(r, n, V), dtype, params(r, n, "mixed"), r.rand(n).astype(np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["", "T", "k", "p", "m", "Tk", "Tp", "Tm", "kp", "pm", "Tkpm"])
def test_sample_each_cut(ctx, kind, dtype):
    r = np.random.RandomState(len(kind) + 10)
    check_sample(ctx, rows(r, 24, 5003), dtype, params(r, 24, kind), r.rand(24).astype(np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,n", [(128256, 6), (152064, 5), (131071, 4), (1 << 20, 2)])
def test_sample_large_vocabularies(ctx, V, n, dtype):
    r = np.random.RandomState(n)
    check_sample(ctx, rows(r, n, V), dtype, params(r, n, "Tp"), r.rand(n).astype(np.float32))
    check_sample(ctx, rows(r, n, V), dtype, params(r, n, "mixed"), r.rand(n).astype(np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("stride,misalign", [(2003, 0), (2008, 0), (2001, 1), (4096, 3)])
def test_sample_strides_and_alignment(ctx, stride, misalign, dtype):
    r = np.random.RandomState(stride)
    check_sample(ctx, rows(r, 9, 2001), dtype, params(r, 9, "mixed"), r.rand(9).astype(np.float32),
                 stride=stride, misalign=misalign)


def test_a_strided_view_is_taken_as_it_is(ctx):
    r = np.random.RandomState(3)
    x = rows(r, 5, 700)
    q, u = params(r, 5, "mixed"), r.rand(5).astype(np.float32)
    want, _ = run_sample(ctx, x, F32, q, u)
    wide = torch.full((5, 720), float("nan"), device="cuda")
    wide[:, 9:709] = dev(x)
    tok = torch.zeros(5, dtype=torch.int32, device="cuda")
    sv.specverify_sample_filtered(ctx, None, F32, 5, 700, 720, filt(q), wide[:, 9:709], dev(u), tok)
    assert np.array_equal(tok.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_ties(ctx, dtype):
    """Few distinct values: most cuts fall inside a run of equal values, where the lowest ids
    stay.  Weights are powers of 2, so that sums are exact on both sides."""
    r = np.random.RandomState(8)
    n, V = 64, 3001
    x = (-r.randint(0, 6, (n, V))).astype(np.float32)
    q = dict(T=np.full(n, 1.4426950408889634, np.float32), k=r.randint(1, 2500, n).astype(np.int32),
             p=r.uniform(0.05, 1, n).astype(np.float32), m=np.zeros(n, np.float32))
    check_sample(ctx, x, dtype, q, r.rand(n).astype(np.float32))
    q["k"][:] = 0
    q["m"] = r.choice([0.0, 0.1, 0.3, 1.0], n).astype(np.float32)
    check_sample(ctx, x, dtype, q, r.rand(n).astype(np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("value", [0.0, -0.0, 5.5, -3.0e38, 1e-30, 700.0, -1000.0])
def test_sample_equal_rows(ctx, value, dtype):
    """Every id has weight 1: the kept ids and the draw are exact in integers."""
    r = np.random.RandomState(2)
    n, V = 10, 20011
    q = params(r, n, "kp")
    q["k"][::2] = 0
    x = np.full((n, V), value, np.float32)
    u = (r.randint(0, 1 << 23, n) / float(1 << 23)).astype(np.float32)
    _, val = as_dtype(x, dtype)
    g, gp = run_sample(ctx, as_dtype(x, dtype)[0], dtype, q, u)
    for i in range(n):
        k = int(q["k"][i]) or V
        kept = max(1, int(np.ceil(float(q["p"][i]) * k)))
        assert g[i] == int(np.floor(float(u[i]) * kept)) and gp[i] == np.float32(1.0 / kept)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("low", [-np.inf, -3.3895313892515355e38, -1e9, -300.0])
@pytest.mark.parametrize("left", [1, 3, 900])
def test_sample_masked_ids(ctx, low, left, dtype):
    """All but `left` ids masked out, by -inf or by a low value; k may pass what is left."""
    r = np.random.RandomState(left)
    n, V = 16, 9001
    x = np.full((n, V), low, np.float32)
    for i in range(n):
        x[i, r.permutation(V)[:left]] = r.standard_normal(left) * 2
    q = params(r, n, "mixed")
    q["k"][1] = 5000
    q["p"][1] = 1.0
    check_sample(ctx, x, dtype, q, r.rand(n).astype(np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1e-30, 1e-7, 1e-3, 40.0, 500.0, 1e5, 1e37])
def test_sample_scales(ctx, scale, dtype):
    """Logits far smaller and far larger than usual, some exactly zero of either sign."""
    r = np.random.RandomState(4)
    n, V = 12, 6007
    x = rows(r, n, V, scale)
    x[:, ::97] = 0.0
    x[:, ::101] = -0.0
    check_sample(ctx, x, dtype, params(r, n, "mixed"), r.rand(n).astype(np.float32))
    q = params(r, n, "kp")
    q["T"] = np.full(n, scale, np.float32)
    check_sample(ctx, x, dtype, q, r.rand(n).astype(np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift", [-200.0, 180.0, 250.0])
def test_sample_shifted_rows(ctx, shift, dtype):
    """A law does not change with a shift of its row: rows far from zero, across the powers of 2."""
    r = np.random.RandomState(6)
    check_sample(ctx, rows(r, 12, 7001, 9.0) + np.float32(shift), dtype, params(r, 12, "mixed"),
                 r.rand(12).astype(np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_peaked_rows(ctx, dtype):
    """One id far above a tail that still counts for the nucleus."""
    r = np.random.RandomState(12)
    n, V = 16, 30011
    x = rows(r, n, V, 1.0)
    x[np.arange(n), r.randint(0, V, n)] = r.uniform(6, 25, n)
    for kind in ("p", "kp", "m", ""):
        check_sample(ctx, x, dtype, params(r, n, kind), r.rand(n).astype(np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_ends_of_the_uniform(ctx, dtype):
    """u = 0 takes the first kept id of positive weight, u = 1 the last."""
    r = np.random.RandomState(1)
    n, V = 8, 4000
    x = rows(r, n, V)
    x[:, :50] = -np.inf
    q = params(r, n, "k")
    bits, val = as_dtype(x, dtype)
    for u, pick in ((0.0, 0), (1.0, -1)):
        g, _ = run_sample(ctx, bits, dtype, q, np.full(n, u, np.float32))
        for i in range(n):
            kept = np.flatnonzero(model.law(val[i], 1.0, int(q["k"][i]))[0] > 0)
            assert g[i] == kept[pick]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_rows_without_a_law(ctx, dtype):
    """NaN, +inf, nothing finite, or parameters out of range: -1 and NaN for that row alone."""
    r = np.random.RandomState(7)
    n, V = 20, 3333
    x = rows(r, n, V)
    q = params(r, n, "mixed")
    x[0, 17], x[1, V - 1], x[2, 0] = np.nan, np.inf, -np.nan
    x[3], x[4] = -np.inf, np.nan
    for i, (c, v) in enumerate([("T", -1), ("T", np.nan), ("T", np.inf), ("p", -0.1), ("p", 1.01),
                                ("p", np.nan), ("m", -0.5), ("m", 1.5), ("m", np.nan)]):
        q[c][5 + i] = v
    u = r.rand(n).astype(np.float32)
    check_sample(ctx, x, dtype, q, u)
    g, gp = run_sample(ctx, as_dtype(x, dtype)[0], dtype, q, u)
    assert np.all(g[:14] == -1) and np.all(np.isnan(gp[:14])) and np.all(g[14:] >= 0)


def test_absent_arrays_cut_nothing(ctx):
    """No filter at all is the plain sampler's law."""
    r = np.random.RandomState(9)
    n, V = 32, 12007
    x, u = rows(r, n, V), r.rand(n).astype(np.float32)
    d, du = dev(x), dev(u)
    tok = torch.zeros(3, n, dtype=torch.int32, device="cuda")
    pr = torch.zeros(3, n, device="cuda")
    sv.specverify_sample(ctx, None, F32, n, V, 1.0, d, du, tok[0], pr[0])
    sv.specverify_sample_filtered(ctx, None, F32, n, V, V, None, d, du, tok[1], pr[1])
    sv.specverify_sample_filtered(ctx, None, F32, n, V, V, sv.SpecVerifyFilter(), d, du, tok[2], pr[2])
    t = tok.cpu().numpy()
    assert np.array_equal(t[1], t[2])
    want, prob, mar = model.sample(x, u, *(params(r, n, "")[c] for c in "Tkpm"))
    assert np.array_equal(t[1], want)
    assert np.array_equal(t[0][mar > 1e-6], want[mar > 1e-6])
    np.testing.assert_allclose(pr[0].cpu(), pr[1].cpu(), rtol=1e-5)


# ------------------------------------------------------------------------------ verify

def run_verify(ctx, tgt, drf, dtype, ft, fd, x, u, probs=True, stream=None, misalign=0):
    B, K1, V = tgt.shape
    K = K1 - 1
    put = (lambda a: dev_offset(a, misalign)) if misalign else dev
    acc = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    out = torch.full((B, K + 1), -7, dtype=torch.int32, device="cuda")
    pr = torch.full((B, K, 2), -7.0, device="cuda") if probs else None
    sv.specverify_run_sampling_filtered(ctx, stream, dtype, B, K, V, filt(ft),
                                        None if fd is None else filt(fd), put(tgt),
                                        put(drf) if K else None, dev(x) if K else None, dev(u), acc,
                                        out, pr if K else None)
    torch.cuda.synchronize()
    return acc.cpu().numpy(), out.cpu().numpy(), None if pr is None else pr.cpu().numpy()


def workload(r, B, K, V, dtype, ft, fd, noise=0.4, scale=3.0):
    t = rows(r, B * (K + 1), V, scale).reshape(B, K + 1, V)
    d = t[:, :K] + rows(r, B * K, V, noise).reshape(B, K, V)
    tb, tv = as_dtype(t, dtype)
    db, dv = as_dtype(d, dtype)
    x = np.zeros((B, K), np.int32)
    for b in range(B):
        for j in range(K):
            q = model.law(dv[b, j], fd["T"][b], int(fd["k"][b]), fd["p"][b], fd["m"][b])[0]
            x[b, j] = r.choice(V, p=q / q.sum())
    return tb, tv, db, dv, x, r.rand(B, K + 1).astype(np.float32)


def check_verify(ctx, w, dtype, ft, fd, same=False, **kw):
    tb, tv, db, dv, x, u = w
    acc, out, prob, mar = model.verify(tv, dv, x, u, ft, fd)
    clear = mar > model.CLEAR
    assert clear.mean() > 0.85
    g = run_verify(ctx, tb, db, dtype, ft, None if same else fd, x, u, **kw)
    assert np.array_equal(g[0][clear], acc[clear]), (g[0], acc)
    assert np.array_equal(g[1][clear], out[clear])
    if g[2] is not None:
        np.testing.assert_allclose(g[2][clear], prob[clear], rtol=PROB_RTOL, atol=2.0 ** -149)
    return acc


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,K,V", [(1, 1, 1), (1, 4, 1000), (3, 1, 2), (5, 2, 63), (7, 5, 1025),
                                   (4, 8, 8193), (2, 3, 50257), (3, 0, 999), (2, 63, 257)])
def test_verify_sizes(ctx, B, K, V, dtype):
    r = np.random.RandomState(B * 1000 + K)
    f = params(r, B, "mixed")
    check_verify(ctx, workload(r, B, K, V, dtype, f, f), dtype, f, f, same=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["", "k", "p", "m", "Tkpm", "mixed"])
def test_verify_each_cut_with_a_draft_filter_of_its_own(ctx, kind, dtype):
    r = np.random.RandomState(len(kind))
    ft, fd = params(r, 24, kind), params(r, 24, "mixed")
    acc = check_verify(ctx, workload(r, 24, 4, 3003, dtype, ft, fd), dtype, ft, fd)
    assert len(set(acc.tolist())) >= 3          # rejections at several places


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_verify_with_ties_at_the_cut(ctx, dtype):
    """Laws of few distinct values: whether a draft id is kept depends on its rank among equals."""
    r = np.random.RandomState(5)
    B, K, V = 32, 4, 2003
    f = dict(T=np.full(B, 1.4426950408889634, np.float32), k=r.randint(100, 1500, B).astype(np.int32),
             p=np.ones(B, np.float32), m=np.zeros(B, np.float32))
    t = (-r.randint(0, 4, (B, K + 1, V))).astype(np.float32)
    d = (-r.randint(0, 4, (B, K, V))).astype(np.float32)
    d[:16] = t[:16, :K]
    x = r.randint(0, V, (B, K)).astype(np.int32)
    u = r.rand(B, K + 1).astype(np.float32)
    tb, tv = as_dtype(t, dtype)
    db, dv = as_dtype(d, dtype)
    check_verify(ctx, (tb, tv, db, dv, x, u), dtype, f, f)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_verify_of_a_draft_equal_to_its_target_accepts_everything(ctx, dtype):
    r = np.random.RandomState(6)
    f = params(r, 12, "mixed")
    acc = check_verify(ctx, workload(r, 12, 3, 5001, dtype, f, f, noise=0.0), dtype, f, f, same=True)
    assert np.all(acc == 3)


def test_verify_bad_sequences_are_marked_alone(ctx):
    r = np.random.RandomState(11)
    B, K, V = 9, 3, 1501
    f = params(r, B, "kp")
    tb, tv, db, dv, x, u = workload(r, B, K, V, F32, f, f)
    x[0, 1], x[1, 2] = -1, V
    tb[2, 3, 7], tb[3, 0, :], db[4, 2, 5] = np.nan, -np.inf, np.inf
    f["p"][5] = 1.5
    acc = check_verify(ctx, (tb, tb, db, db, x, u), F32, f, f)
    assert np.all(acc[:6] == -1) and np.all(acc[6:] >= 0)


def test_verify_rows_off_alignment_and_without_probabilities(ctx):
    r = np.random.RandomState(13)
    f = params(r, 6, "mixed")
    check_verify(ctx, workload(r, 6, 3, 1237, BF16, f, f), BF16, f, f, misalign=3, probs=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_verify_served_shape(ctx, dtype):
    r = np.random.RandomState(21)
    f = params(r, 8, "mixed")
    check_verify(ctx, workload(r, 8, 4, 128256, dtype, f, f), dtype, f, f, same=True)


def test_verify_law_of_the_emitted_token(ctx):
    """Draft from the cut draft law, verify, emit: over many sequences the first emitted token
    follows the cut target law (the point of verifying with the cut laws).  Each id's count is
    binomial; 6 standard deviations over 40 ids."""
    r = np.random.RandomState(17)
    B, V = 512, 60
    n = 40
    t, d = rows(r, 1, V, 1.5)[0], rows(r, 1, V, 1.5)[0]
    one = dict(T=0.9, k=12, p=0.95, m=0.01)
    f = {c: np.full(B, one[c]).astype(np.int32 if c == "k" else np.float32) for c in one}
    P = model.law(t, *(f[c][0] for c in "Tkpm"))[0]
    Q = model.law(d, *(f[c][0] for c in "Tkpm"))[0]
    count = np.zeros(V)
    for _ in range(n):
        x = r.choice(V, size=(B, 1), p=Q).astype(np.int32)
        u = r.rand(B, 2).astype(np.float32)
        _, out, _ = run_verify(ctx, np.tile(t, (B, 2, 1)), np.tile(d, (B, 1, 1)), F32, f, None, x, u)
        count += np.bincount(out[:, 0], minlength=V)
    sd = np.sqrt(B * n * P * (1 - P))
    assert np.all(np.abs(count - B * n * P) <= 6 * sd + 1e-9)


# ------------------------------------------------------------------------------ calls

def test_capacity_and_argument_errors(ctx):
    small = sv.specverify_create(0, 4, 2, 1000)
    z = torch.zeros(8, 1000, device="cuda")
    u, t = torch.zeros(16, device="cuda"), torch.zeros(16, dtype=torch.int32, device="cuda")

    def status(fn, *a):
        with pytest.raises(sv.SpecVerifyError) as e:
            fn(*a)
        return e.value.status

    s = sv.specverify_sample_filtered
    a = lambda n, V, st, dt=F32: (small, None, dt, n, V, st, None, z.data_ptr(), u, t)
    assert status(s, *a(5, 1000, 1000)) == sv.SPECVERIFY_ECAPACITY
    assert status(s, *a(1, 1001, 1001)) == sv.SPECVERIFY_ECAPACITY
    assert status(s, *a(2, 1000, 999)) == sv.SPECVERIFY_EINVAL
    assert status(s, *a(2, 1000, 1 << 62)) == sv.SPECVERIFY_EINVAL
    assert status(s, *a(2, 1000, 1000, 7)) == sv.SPECVERIFY_EUNSUPPORTED
    assert status(s, small, None, F32, -1, 10, 10, None, z, u, t) == sv.SPECVERIFY_EINVAL
    assert status(s, small, None, F32, 1, 10, 10, None, z.data_ptr() + 2, u, t) == sv.SPECVERIFY_EINVAL
    assert status(s, small, None, F32, 1, 10, 10, None, None, u, t) == sv.SPECVERIFY_EINVAL
    f = sv.SpecVerifyFilter(temperature=u.data_ptr() + 1)
    assert status(s, small, None, F32, 1, 10, 10, f, z, u, t) == sv.SPECVERIFY_EINVAL
    s(small, None, F32, 0, 10, 10, None, None, None, None)          # nothing to do
    v = sv.specverify_run_sampling_filtered
    assert status(v, small, None, F32, 5, 1, 10, None, None, z, z, t, u, t, t) == \
        sv.SPECVERIFY_ECAPACITY
    assert status(v, small, None, F32, 1, 1, 10, None, None, z, None, t, u, t, t) == \
        sv.SPECVERIFY_EINVAL
    sv.specverify_destroy(small)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_replays_of_a_captured_draw_and_verify(ctx, dtype):
    """A sampler and a verify captured into one graph, replayed on new inputs with eager calls
    between the replays: every replay equals the eager result."""
    r = np.random.RandomState(31)
    B, K, V = 6, 3, 9001
    f = params(r, B, "mixed")
    tb, _, db, _, x, u = workload(r, B, K, V, dtype, f, f)
    d = dict(t=dev(tb), d=dev(db), x=dev(x), u=dev(u))
    ff = filt(f)
    c2 = sv.specverify_create(0, B, K, V)
    mk = lambda: (torch.zeros(B, dtype=torch.int32, device="cuda"),
                  torch.zeros(B, K + 1, dtype=torch.int32, device="cuda"),
                  torch.zeros(B, K, 2, device="cuda"),
                  torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, device="cuda"))

    def go(o, handle):
        sv.specverify_run_sampling_filtered(handle, None, dtype, B, K, V, ff, None, d["t"], d["d"],
                                            d["x"], d["u"], o[0], o[1], o[2])
        sv.specverify_sample_filtered(handle, None, dtype, B, V, (K + 1) * V, ff, d["t"], d["u"],
                                      o[3], o[4])

    eager, rep = mk(), mk()
    go(rep, c2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(rep, c2)
    for step in range(4):
        d["u"].copy_(torch.rand(B, K + 1, device="cuda"))
        d["t"].copy_(d["t"].roll(step, -1))
        go(eager, ctx)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, rep):
            assert torch.equal(a, b)
    sv.specverify_destroy(c2)


def test_two_contexts_on_two_streams(ctx):
    r = np.random.RandomState(33)
    B, K, V = 8, 2, 30001
    f = params(r, B, "mixed")
    tb, tv, db, dv, x, u = workload(r, B, K, V, F32, f, f)
    want = run_verify(ctx, tb, db, F32, f, None, x, u)
    other = sv.specverify_create(0, B, K, V)
    ff, args = filt(f), (dev(tb), dev(db), dev(x), dev(u))
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [(torch.zeros(B, dtype=torch.int32, device="cuda"),
             torch.zeros(B, K + 1, dtype=torch.int32, device="cuda"),
             torch.zeros(B, K, 2, device="cuda")) for _ in s]
    torch.cuda.synchronize()
    for _ in range(5):
        for h, st, o in zip((ctx, other), s, outs):
            sv.specverify_run_sampling_filtered(h, st, F32, B, K, V, ff, None, *args, *o)
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, want):
            assert np.array_equal(a.cpu().numpy(), b, equal_nan=True)
    sv.specverify_destroy(other)
