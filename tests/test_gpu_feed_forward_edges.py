"""The feed-forward block where its kernels change shape and where values leave their range, against its 64-bit
statement (oracle/token_rows.py).  The helpers and how their tolerances are derived: test_gpu_feed_forward.py."""
import math

import numpy as np
import pytest
import torch

from oracle import token_rows as ref
from tests.test_gpu_feed_forward import ALL, H, TINY, U, check, f64, gen, placed, routed, weights, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spmv():
    import __graft_entry__

    __graft_entry__._build_module().build()
    import sparse_matrix_vector_csr_gb300 as spmv

    return spmv


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,experts", [(1, None), (8, None), (9, None), (16, None), (17, None), (200, None), (20, 8), (50, 8), (400, 8)])
def test_infinite_weights(spmv, dtype, rows, experts):
    """an infinity in w_down gives infinities of the sign of h (NaN where two meet), as many rows as there are"""
    g = gen(rows)
    d, f = 72, 136
    if experts is None:
        x, run = torch.randn(rows, d, generator=g).to(dtype).cuda(), spmv.feed_forward
        spans = [(0, rows)]
    else:
        plan, x, _, spans = routed(spmv, rows, 1, experts, 1, d, dtype, g, dropped=0.0)
        run = plan.feed_forward
    wg, wu, wd = weights(experts, d, f, dtype, g)
    clean = run(x, wg, wu, wd)
    bad = wd.clone()
    bad[..., 3, 5], bad[..., 4, 7], bad[..., 6, 9], bad[..., 6, 10] = math.inf, -math.inf, math.inf, -math.inf
    y = f64(run(x, wg, wu, bad).y)
    hit = np.array([3, 4, 6])
    for e, (a, b) in enumerate(spans):
        w = [f64(t if experts is None else t[e]) for t in (wg, wu, bad)]
        xe = f64(x[a:b])
        h = ref.act(xe @ w[0].T, "silu")[0] * (xe @ w[1].T)
        sure = (np.abs(h[:, [5, 7, 9, 10]]) > 1e-4).all(1)  # (no rounding moves one across 0)
        assert 2 * sure.sum() >= b - a
        with np.errstate(invalid="ignore"):
            want = h @ w[2].T
        assert np.array_equal(y[a:b][sure][:, hit], want[sure][:, hit], equal_nan=True), (e, y[a:b][:, hit], want[:, hit])
    rest = [c for c in range(d) if c not in hit]
    assert np.array_equal(y[:, rest], f64(clean.y)[:, rest])
