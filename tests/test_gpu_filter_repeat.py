"""The same call gives the same result: rows whose halves hold the same values in other orders, drawn
at one half, so that which half the draw falls into hangs on the last bit of its sums."""
import numpy as np
import pytest
import torch

from gpu_support import dev
from rejection_sampling_verification_row_amd import binding as sv
from test_gpu_filter import BF16, F32, as_dtype, ctx, filt, rows  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [32000, 128256])
@pytest.mark.parametrize("cut", [dict(k=50), dict(k=900), dict(m=1e-4), dict(m=0.02), dict(k=900, m=0.02)])
def test_draws_at_the_edge_of_rounding_repeat(ctx, cut, V, dtype):
    r = np.random.RandomState(V)
    n = 128
    half = rows(r, n, V // 2)
    x = np.concatenate([half, np.stack([r.permutation(h) for h in half])], axis=1)
    q = dict(T=np.ones(n, np.float32), k=np.full(n, cut.get("k", 0), np.int32),
             p=np.ones(n, np.float32), m=np.full(n, cut.get("m", 0), np.float32))
    d, f, u = dev(as_dtype(x, dtype)[0]), filt(q), torch.full((n,), 0.5, device="cuda")
    tok = torch.zeros(40, n, dtype=torch.int32, device="cuda")
    for t in tok:
        sv.specverify_sample_filtered(ctx, None, dtype, n, V, V, f, d, u, t)
    t = tok.cpu().numpy()
    assert np.all(t >= 0) and np.all(t == t[0]), (t != t[0]).any(0).sum()
