"""The sparse-row operators on the GPU against their 64-bit statements (oracle/sparse_rows.py).

Tolerances come from the arithmetic: E = 2^-24 is half a unit of a float, H[dtype] that of the
output's type; a hardware 2^x is within 2^-22, its argument (a difference, scaled) within 3 E of
itself, and sums run over at most a few hundred terms one after the other before trees.
"""
import math

import numpy as np
import pytest
import torch

from oracle import sparse_rows as ref

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
H = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-37}  # subnormal outputs, flushed exponentials
SUM = 2e-5  # relative error of a sum of exponentials: 2^-22 and 3 E |x| exp(-|x|) a term, up to 300 E of summing
ALL = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def spmv():
    import __graft_entry__

    __graft_entry__._build_module().build()
    import sparse_matrix_vector_csr_gb300 as spmv

    return spmv


def placed(t, shift=0, pad=0):
    """The matrix t at an address `shift` values behind an aligned one, rows `pad` values apart,
    NaN around them."""
    rows, n = t.shape
    buf = torch.full((shift + rows * (n + pad) + 8,), math.nan, dtype=t.dtype, device="cuda")
    view = buf[shift:shift + rows * (n + pad)].view(rows, n + pad)[:, :n]
    view.copy_(t)
    return view, buf


def surroundings_untouched(view, buf):
    inside = torch.zeros_like(buf, dtype=torch.bool)
    torch.as_strided(inside, view.shape, view.stride(), view.storage_offset()).fill_(True)
    return bool(torch.isnan(buf[~inside]).all())


def f64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    return torch.Generator().manual_seed(seed)


# --------------------------------------------------------------------------- #
# the k largest entries of each row
# --------------------------------------------------------------------------- #


def check_top(spmv, x, k, tau=1.0, weighting="row"):
    top = spmv.topk_rows(x, k, temperature=tau, weights=weighting, lse=True, vals=True)
    ids, vals, w, lse = top.ids.cpu().numpy(), f64(top.vals), f64(top.weights), f64(top.lse)
    for r, row in enumerate(f64(x)):
        i, v = ref.topk_row(row, k)
        assert np.array_equal(ids[r], i), (r, ids[r], i)
        assert np.array_equal(vals[r], v, equal_nan=True)
        norm = ref.lse(row / tau)
        if np.isfinite(norm):
            assert abs(lse[r] - norm) <= SUM + 4 * E * (abs(norm) + np.abs(row[i[0]]) / tau)
        elif not np.isnan(row).any():
            assert lse[r] == norm or np.isnan(norm) and np.isnan(lse[r])
        want = ref.top_weights(row, i, v, weighting, tau)
        if np.isfinite(want).all():
            # the argument's own rounding counts relative to the weight
            np.testing.assert_allclose(w[r], want, rtol=2 * SUM + 8 * E * np.nanmax(np.abs(v[np.isfinite(v)] / tau), initial=0),
                                       atol=1e-37)
    return top


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,n,k", [(1, 1, 1), (3, 2, 2), (9, 7, 3), (8, 64, 4), (5, 100, 32), (33, 256, 8),
                                      (4, 512, 16), (3, 513, 8), (2, 300, 33), (3, 1000, 256), (2, 1500, 256), (200, 5000, 200), (2, 4097, 64),
                                      (1, 50021, 200), (3, 33000, 1), (1, 131072, 64), (2, 70001, 128),
                                      (1, 262144, 50), (1, 300001, 20), (1, 700003, 256)])
def test_topk_rows(spmv, dtype, rows, n, k):
    x = (torch.randn(rows, n, generator=gen(n + k)) * 3).to(dtype).cuda()
    check_top(spmv, x, k, weighting="row")
    check_top(spmv, x, k, tau=0.7, weighting="selected")


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("n", [64, 2000, 40000])
@pytest.mark.parametrize("shift,pad", [(1, 0), (3, 5), (0, 8)])
def test_topk_rows_any_address(spmv, dtype, n, shift, pad):
    x, _ = placed((torch.randn(3, n + 1, generator=gen(n)) * 2).to(dtype), shift, pad)
    check_top(spmv, x, 9)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("n", [40, 3000, 150000])
def test_topk_rows_ties_masks_and_extremes(spmv, dtype, n):
    low = torch.finfo(dtype).min
    x = torch.zeros(12, n, dtype=torch.float32)
    x[1] = torch.arange(n) % 3                                    # ties across the whole row
    x[2] = -math.inf                                              # nothing to take
    x[3] = -math.inf
    x[3, [n - 1, n // 2, 5]] = torch.tensor([-7.0, 2.0, -7.0])    # fewer than k
    x[4] = low                                                    # the lowest value is a value
    x[5] = low
    x[5, n // 3] = 1.0
    x[6] = torch.arange(n) / n                                    # ascending
    x[7] = -torch.arange(n) / n - 300.0                           # descending, far below 0
    x[8, n // 2] = math.inf
    x[9, [1, n - 2]] = math.nan
    x[10] = -0.0
    x[10, n // 2:] = 0.0                                          # -0 and +0 are equal
    x[11, : min(n, 2500)] = 5.0                                   # more ties on top than candidates
    x = x.to(dtype).cuda()
    for k in (1, 8, 30):
        check_top(spmv, x, k)
    nan = torch.full((2, n), math.nan, dtype=dtype).cuda()
    assert spmv.topk_rows(nan, 3).ids.tolist() == [[0, 1, 2]] * 2


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,n,k", [(5, 8, 3), (40, 256, 8), (3, 1500, 20), (2, 33001, 64)])
@pytest.mark.parametrize("weighting", ["selected", "row"])
@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 3)])
def test_topk_rows_grad(spmv, dtype, rows, n, k, weighting, shift, pad):
    g = gen(rows + n)
    x = (torch.randn(rows, n, generator=g) * 2)
    x[torch.rand(rows, n, generator=g) < 0.1] = -math.inf
    x[0] = -math.inf
    x[-1, 1:] = -math.inf
    x, _ = placed(x.to(dtype), shift, pad)
    tau = 1.5
    top = spmv.topk_rows(x, k, temperature=tau, weights=weighting)
    dw = torch.randn(rows, k, generator=g).cuda()
    other, buf = placed(torch.zeros(rows, n, dtype=dtype), shift + 1, pad + 2)  # at another offset than x
    top.grad(dw, out=other)
    assert surroundings_untouched(other, buf)
    out, buf = placed(torch.zeros(rows, n, dtype=dtype), shift, pad)
    assert top.grad(dw, out=out) is out
    assert surroundings_untouched(out, buf)
    assert torch.equal(out, other)
    ids, w, d = top.ids.cpu().numpy(), f64(top.weights), f64(dw)
    for r, row in enumerate(f64(x)):
        want = ref.top_weights_grad(row, ids[r], w[r], d[r], weighting, tau)
        # w's own error enters: 2 SUM of every product and of their sum
        size = np.zeros(n)
        live = ids[r] >= 0
        q = np.exp(row / tau - ref.lse(row / tau)) if weighting == "row" and live.any() else np.zeros(n)
        dot = np.abs(w[r] * d[r]).sum()
        size += q * dot
        size[ids[r][live]] += (np.abs(w[r] * d[r]) + w[r] * dot)[live]
        np.testing.assert_array_less(np.abs(f64(out[r]) - want), 4 * SUM * size / tau + H[dtype] * np.abs(want) + TINY[dtype])


# --------------------------------------------------------------------------- #
# rows sorted by expert and back
# --------------------------------------------------------------------------- #


def some_ids(tokens, k, experts, g, dropped=0.1):
    """k distinct experts a token, some liked, some entries dropped, token 1 without any."""
    score = torch.rand(tokens, experts, generator=g) + 0.5 * torch.rand(1, experts, generator=g)
    ids = score.topk(min(k, experts), dim=1).indices.to(torch.int32)
    if k > experts:
        ids = ids.repeat(1, -(-k // experts))[:, :k]
    ids[torch.rand(tokens, k, generator=g) < dropped] = -1
    if tokens > 1:
        ids[1] = -1
    return ids.contiguous()


def check_plan(spmv, ids, experts, align):
    plan = spmv.RoutePlan(ids.cuda(), experts, align)
    offsets, slots, sources = ref.route_plan(ids.numpy(), experts, align, plan.rows)
    assert plan.offsets.cpu().numpy().tolist() == offsets.tolist()
    assert np.array_equal(plan.slots.cpu().numpy(), slots)
    assert np.array_equal(plan.sources.cpu().numpy(), sources)
    return plan, slots, sources


@pytest.mark.parametrize("tokens,k,experts,align", [
    (0, 2, 4, 8), (1, 1, 1, 1), (1, 8, 128, 1), (4, 8, 128, 16), (33, 3, 17, 16), (1000, 2, 4, 128), (700, 3, 600, 1),
    (513, 4, 4096, 2), (3000, 8, 64, 1), (20000, 8, 128, 128), (40000, 8, 7, 5), (5, 6, 3, 4), (2049, 1, 2, 1)])
def test_route_plan(spmv, tokens, k, experts, align):
    ids = some_ids(tokens, k, experts, gen(tokens + k))
    check_plan(spmv, ids, experts, align)


def test_route_plan_extremes(spmv):
    for ids in (torch.full((3000, 2), -1), torch.zeros(3000, 2), torch.full((3000, 2), 9),
                torch.tensor([[2 ** 31 - 1, -2 ** 31], [8, 9], [0, 0]])):
        check_plan(spmv, ids.to(torch.int32), 9, 32)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("tokens,k,experts,align,d", [
    (1, 1, 1, 1, 1), (1, 8, 16, 1, 4096), (4, 8, 128, 4, 256), (7, 3, 5, 16, 77), (300, 2, 9, 1, 1537),
    (65, 5, 30, 8, 132), (40, 9, 12, 1, 2050), (33, 33, 40, 1, 64), (3, 2, 4, 64, 9000)])
def test_route_rows(spmv, dtype, tokens, k, experts, align, d):
    g = gen(tokens * d)
    ids = some_ids(tokens, k, experts, g)
    plan, slots, sources = check_plan(spmv, ids, experts, align)

    def rand(rows):
        return torch.randn(rows, d, generator=g).to(dtype)

    for shift, pad in ((0, 0), (1, 0), (2, 6)):
        x, _ = placed(rand(tokens), shift, pad)
        ys, _ = placed(rand(plan.rows), shift, pad)
        ys[torch.from_numpy(sources < 0).cuda()] = math.nan  # rows that no entry has are not read
        w = torch.randn(tokens, k, generator=g).cuda()
        w[torch.from_numpy(slots < 0).cuda()] = math.nan
        xs_out, xs_buf = placed(torch.zeros(plan.rows, d, dtype=dtype), shift, pad)
        y_out, y_buf = placed(torch.zeros(tokens, d, dtype=dtype), shift, pad)
        dys_out, dys_buf = placed(torch.zeros(plan.rows, d, dtype=dtype), shift, pad)
        xs_out.fill_(math.nan), y_out.fill_(math.nan), dys_out.fill_(math.nan)
        xs = plan.dispatch(x, out=xs_out)
        assert np.array_equal(f64(xs), ref.dispatch(f64(x), slots, plan.rows))
        y = plan.combine(ys, w, out=y_out)
        want = ref.combine(f64(ys), slots, f64(w))
        size = ref.combine(np.abs(f64(ys)), slots, np.abs(f64(w)))
        assert (np.abs(f64(y) - want) <= (k + 1) * E * size + H[dtype] * np.abs(want) * 1.01 + TINY[dtype]).all()
        dys, dw = plan.combine_grad(x, ys, w, out=dys_out)
        want_dys, want_dw = ref.combine_grad(f64(x), f64(ys), slots, f64(w))
        assert (np.abs(f64(dys) - want_dys) <= (E + H[dtype]) * 1.01 * np.abs(want_dys) + TINY[dtype]).all()
        size = ref.combine_grad(np.abs(f64(x)), np.abs(f64(ys)), slots, f64(w))[1]
        # one thread adds at most 8 (d / 2048 + 1) products, then trees of 5 and 8 levels
        assert (np.abs(f64(dw) - want_dw) <= (8 * (d // 256 + 1) + 16) * E * size).all()
        dx = plan.dispatch_grad(ys)
        want = ref.combine(f64(ys), slots, None)
        size = ref.combine(np.abs(f64(ys)), slots, None)
        assert (np.abs(f64(dx) - want) <= (k + 1) * E * size + H[dtype] * np.abs(want) * 1.01 + TINY[dtype]).all()
        for view, buf in ((xs_out, xs_buf), (y_out, y_buf), (dys_out, dys_buf)):
            assert surroundings_untouched(view, buf)


def test_route_rows_past_32_bits(spmv):
    """Sorted rows beyond 2^32 bytes and 2^31 values."""
    tokens, d, experts = 70001, 32776, 3
    ids = torch.zeros(tokens, 1, dtype=torch.int32)
    ids[::2] = 2
    plan = spmv.RoutePlan(ids.cuda(), experts)
    x = torch.empty(tokens, d, dtype=torch.bfloat16, device="cuda")
    x[:] = (torch.arange(tokens, device="cuda") % 251).to(torch.bfloat16)[:, None]
    xs = plan.dispatch(x)
    order = torch.cat([torch.arange(1, tokens, 2), torch.arange(0, tokens, 2)]).cuda()
    assert torch.equal(xs[:, 0], x[order, 0]) and torch.equal(xs[:, -1], x[order, -1])
    w = torch.full((tokens, 1), 0.5, device="cuda")
    y = plan.combine(xs, w)
    assert torch.equal(y[:, 5], x[:, 5] * 0.5) and torch.equal(y[-1], x[-1] * 0.5)
    del y
    dys, dw = plan.combine_grad(x, xs, w)
    assert torch.equal(dys[-1], xs[-1] * 0.5)
    assert torch.allclose(dw[:, 0], x[:, 0].float() ** 2 * d, rtol=1e-4)


# --------------------------------------------------------------------------- #
# distillation
# --------------------------------------------------------------------------- #


def some_target(rows, vocab, k, g, absent=0.1):
    ids = torch.stack([torch.randperm(vocab, generator=g)[:k] if vocab * rows < 100000 else
                       torch.randint(0, vocab // k, (k,), generator=g) + torch.arange(k) * (vocab // k)
                       for _ in range(rows)]).to(torch.int32) if rows else torch.zeros(0, k, dtype=torch.int32)
    if ids.shape[1] < k:
        ids = torch.cat([ids, torch.full((rows, k - ids.shape[1]), -1, dtype=torch.int32)], 1)
    ids[torch.rand(rows, k, generator=g) < absent] = -1
    ids[(torch.rand(rows, k, generator=g) < absent / 2) & (ids < 0)] = vocab  # outside: no entry either
    if rows > 2:
        ids[2] = -1
    teacher = torch.randn(rows, k, generator=g) * 2 + 3
    if k > 2:
        teacher[0, 1] = -math.inf
    return ids.contiguous(), teacher


def check_distill(spmv, z, ids, teacher, lse, tau, modes=("fused", "two"), out=None, scale=0.75, teacher_dtype=torch.float32):
    rows, vocab = z.shape
    dtype = z.dtype
    teacher = teacher.to(teacher_dtype)
    zs, ts, i = f64(z), f64(teacher), ids.numpy()
    n = [None] * rows if lse is None else f64(lse)
    args = (z, ids.cuda(), teacher.cuda())
    kw = {"teacher_lse": None if lse is None else lse.cuda(), "temperature": tau}
    want = np.array([ref.distill_loss(zs[r], i[r], ts[r], n[r], tau) for r in range(rows)])
    row_scale = torch.linspace(0.5, 2.0, rows)

    def check_loss(loss):
        for r in range(rows):
            t = ref._target(zs[r], i[r], ts[r], n[r], tau)
            if t is None:
                assert loss[r] == 0.0
                continue
            zz, cols, p, logp, rest, _, lse_rest, norm = t
            m = zz.max()
            live = p > 0
            # p's error: that of its logarithm, whose terms are rounded in 32 bits
            ep = 4 * E * (np.abs(ts[r]).max(initial=0, where=np.isfinite(ts[r])) / tau + (abs(n[r]) if n[r] is not None else 0) + 4) + SUM
            terms = np.abs(logp[live]) + np.abs(zz[cols][live] - m) + abs(norm - m) + 1
            tol = (p[live] * terms).sum() * (ep + 8 * E) + SUM
            if rest > 0:
                # the remainder carries p's absolute error
                tol += (ep * p.sum() + 4 * E) * (abs(np.log(rest)) + 2 + abs(lse_rest - norm)) + rest * 2 * SUM
            assert abs(loss[r] - want[r]) <= tol or (np.isinf(want[r]) and loss[r] == want[r]), (r, loss[r], want[r], tol)

    def check_grad(dz, scales):
        for r in range(rows):
            g = ref.distill_grad(zs[r], i[r], ts[r], n[r], tau) * scales[r]
            t = ref._target(zs[r], i[r], ts[r], n[r], tau)
            if t is None:
                assert not dz[r].any()
                continue
            zz, cols, p, _, rest, others, lse_rest, norm = t
            q = np.exp(zz - norm)
            ep = 4 * E * (np.abs(ts[r]).max(initial=0, where=np.isfinite(ts[r])) / tau + (abs(n[r]) if n[r] is not None else 0) + 4) + SUM
            arg = 4 * E * np.abs(np.where(np.isfinite(zz), zz - zz.max(), 0.0))  # the exponent's rounding
            size = q * (SUM + arg)
            if rest > 0:
                share = np.exp(zz[others] - lse_rest)  # of the other columns' mass
                rel = SUM + 4 * E * np.abs(np.where(np.isfinite(zz[others]), zz[others] - zz[others].max(), 0.0))
                size[others] += share * ((SUM + rel) * rest + ep * p.sum() + 4 * E)
            size[cols] += p * ep
            tol = size * abs(scales[r]) / tau * 1.01 + H[dtype] * 1.01 * np.abs(g) + TINY[dtype]
            bad = np.flatnonzero(~(np.abs(dz[r] - g) <= tol))
            assert bad.size == 0, (r, bad[:5], dz[r][bad[:5]], g[bad[:5]], tol[bad[:5]])

    if "two" in modes:
        res = spmv.distill_loss(*args, **kw)
        check_loss(f64(res.loss))
        dz = res.grad(row_scale.cuda(), scale=scale, out=out)
        check_grad(f64(dz), scale * row_scale.double().numpy())
    if "fused" in modes:
        loss, dz = spmv.distill_loss_grad(*args, **kw, scale=scale, out=out)
        check_loss(f64(loss))
        check_grad(f64(dz), np.full(rows, scale))
        loss2, dz2 = spmv.distill_loss_grad(*args, **kw, scale=scale, row_scale=row_scale.cuda())
        assert torch.equal(loss, loss2)
        check_grad(f64(dz2), scale * row_scale.double().numpy())


def teacher_lse_of(ids, teacher, vocab, tau, g):
    """A log-sum that leaves between 1 % and 40 % of the mass to the other columns."""
    t = torch.where((ids >= 0) & (ids < vocab), teacher.double() / tau, -math.inf)
    lse = torch.logsumexp(t, 1)
    lse = torch.where(torch.isfinite(lse), lse, 0.0)
    return (lse - torch.log1p(-(torch.rand(len(ids), generator=g).double() * 0.39 + 0.01))).float()


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (3, 2, 1), (4, 7, 3), (5, 33, 8), (9, 257, 16), (4, 1000, 33),
                                          (6, 4097, 64), (3, 8192, 512), (3, 20011, 20), (1, 32768, 16), (2, 50021, 64),
                                          (1, 131072, 64), (1, 151937, 100), (1, 262144, 8), (1, 300007, 64),
                                          (1, 600011, 30), (160, 9000, 20), (330, 17001, 64), (153, 70001, 33),
                                          (155, 131072, 64), (200, 33000, 300), (152, 270001, 5), (1300, 40, 5),
                                          (1217, 700, 33), (1250, 2001, 12)])
def test_distill(spmv, dtype, tail, rows, vocab, k):
    g = gen(vocab + k)
    tau = 1.0 if vocab % 2 else 2.0
    ids, teacher = some_target(rows, vocab, k, g, absent=0.0 if k == 1 else 0.1)
    z = (torch.randn(rows, vocab, generator=g) * 2 - 40.0).to(dtype).cuda()  # far from 0
    lse = teacher_lse_of(ids, teacher, vocab, tau, g) if tail else None
    check_distill(spmv, z, ids, teacher, lse, tau)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("shift,pad", [(1, 0), (3, 5), (0, 8)])
@pytest.mark.parametrize("rows,vocab", [(5, 1), (5, 131), (5, 9001), (310, 9001), (1217, 131)])
def test_distill_any_address_and_in_place(spmv, dtype, tail, shift, pad, rows, vocab):
    g = gen(vocab + shift)
    ids, teacher = some_target(rows, vocab, min(6, vocab), g)
    z, _ = placed((torch.randn(rows, vocab, generator=g) * 2).to(dtype), shift, pad)
    lse = teacher_lse_of(ids, teacher, vocab, 1.0, g) if tail else None
    out, buf = placed(torch.zeros(rows, vocab, dtype=dtype), shift, pad)
    check_distill(spmv, z, ids, teacher, lse, 1.0, out=out)
    assert surroundings_untouched(out, buf)
    out, buf = placed(torch.zeros(rows, vocab, dtype=dtype), shift + 1, pad)  # another offset than z's
    check_distill(spmv, z, ids, teacher, lse, 1.0, out=out)
    assert surroundings_untouched(out, buf)
    kw = {"teacher_lse": None if lse is None else lse.cuda()}
    args = (ids.cuda(), teacher.cuda())
    for fused in (True, False):  # in place gives the bits that another output gets
        here, buf = placed(z, shift, pad)
        if fused:
            loss, dz = spmv.distill_loss_grad(z, *args, **kw)
            l2, d2 = spmv.distill_loss_grad(here, *args, **kw, out=here)
        else:
            res = spmv.distill_loss(z, *args, **kw)
            loss, dz = res.loss, res.grad()
            res = spmv.distill_loss(here, *args, **kw)
            l2, d2 = res.loss, res.grad(out=here)
        assert torch.equal(l2, loss) and torch.equal(d2, dz) and d2.data_ptr() == here.data_ptr()
        assert surroundings_untouched(here, buf)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("teacher_dtype", ALL)
@pytest.mark.parametrize("rows,vocab", [(8, 300), (8, 40000), (170, 40000), (1300, 300)])
def test_distill_masks_and_teacher_types(spmv, tail, teacher_dtype, rows, vocab):
    g = gen(vocab)
    k = 12
    ids, teacher = some_target(rows, vocab, k, g)
    teacher = teacher.to(teacher_dtype).float()
    z = torch.randn(rows, vocab, generator=g) * 2
    low = torch.finfo(torch.bfloat16).min
    z[:, vocab // 2:] = -math.inf           # a masked half of the vocabulary ...
    z[1, vocab // 2:] = low                 # ... by the lowest value
    z[3, : vocab // 3] = low
    z[2] = math.nan                         # a row without a target may hold anything
    ids = torch.where(ids >= 0, ids % (vocab // 2), ids)  # the teacher's entries lie in the other half
    for r in range(rows):                   # (distinct still)
        seen = set()
        for j in range(k):
            c = int(ids[r, j])
            if c >= 0 and c in seen:
                ids[r, j] = -1
            seen.add(c)
    ids[3] = torch.where((ids[3] >= 0) & (ids[3] < vocab // 3), -1, ids[3])
    z[4, :] = -1000.0                       # one column has everything
    z[4, ids[4][ids[4] >= 0][:1].long()] = 1000.0
    teacher[5] = -math.inf                  # a target without mass
    lse = teacher_lse_of(ids, teacher, vocab, 1.0, g) if tail else None
    check_distill(spmv, z.to(torch.bfloat16).cuda(), ids, teacher, lse, 1.0, teacher_dtype=teacher_dtype)


def test_distill_gradient_is_the_difference(spmv):
    """The kernel's gradient against central differences of the 64-bit loss."""
    g = gen(3)
    z = torch.randn(2, 37, generator=g) * 2
    ids, teacher = some_target(2, 37, 6, g)
    teacher[0, 1] = 0.5
    for lse in (None, teacher_lse_of(ids, teacher, 37, 1.7, g)):
        _, dz = spmv.distill_loss_grad(z.cuda(), ids.cuda(), teacher.cuda(),
                                       teacher_lse=None if lse is None else lse.cuda(), temperature=1.7)
        for r in range(2):
            def f(v):
                return ref.distill_loss(v, ids[r].numpy(), f64(teacher[r]), None if lse is None else float(lse[r]), 1.7)
            for c in range(37):
                a, b = f64(z[r]), f64(z[r])
                a[c] += 1e-5
                b[c] -= 1e-5
                assert abs((f(a) - f(b)) / 2e-5 - float(dz[r, c])) < 2e-5


@pytest.mark.parametrize("rows,vocab", [(1, 1 << 22), (60, 1 << 22), (153, 1000003)])
def test_distill_largest_vocabularies(spmv, rows, vocab):
    g = gen(vocab)
    z = torch.randn(rows, vocab, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    ids, teacher = some_target(rows, vocab, 7, g)
    lse = teacher_lse_of(ids, teacher, vocab, 1.0, g)
    loss, dz = spmv.distill_loss_grad(z, ids.cuda(), teacher.cuda(), teacher_lse=lse.cuda())
    res = spmv.distill_loss(z, ids.cuda(), teacher.cuda(), teacher_lse=lse.cuda())
    assert torch.isfinite(loss).all() and torch.isfinite(dz).all()
    torch.testing.assert_close(res.loss, loss, rtol=1e-4, atol=1e-4)
    for r in (0, rows - 1):
        check_distill(spmv, z[r:r + 1], ids[r:r + 1], teacher[r:r + 1], lse[r:r + 1], 1.0, modes=("fused",))
        want = ref.distill_loss(f64(z[r]), ids[r].numpy(), f64(teacher[r]), float(lse[r]))
        assert abs(float(loss[r]) - want) < 1e-3 * (1 + abs(want))


def test_distill_whole_vocabulary_as_entries(spmv):
    """With every column an entry there is no other class, whatever rounding leaves of r."""
    g = gen(4)
    z = torch.randn(3, 50, generator=g)
    t = torch.randn(3, 50, generator=g)
    ids = torch.arange(50, dtype=torch.int32).repeat(3, 1)
    lse = torch.logsumexp(t.double(), 1).float() + 1e-6
    check_distill(spmv, z.cuda(), ids, t, lse, 1.0)
    # the student has no mass on the others, the teacher nothing but rounding
    z[:, 40:] = -math.inf
    res = spmv.distill_loss(z.cuda(), ids[:, :40].contiguous().cuda(), t[:, :40].contiguous().cuda(),
                            teacher_lse=(torch.logsumexp(t[:, :40].double(), 1).float() + 2e-6).cuda())
    assert torch.isfinite(res.loss).all() and torch.isfinite(res.grad()).all()


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows", [3, 1300])
def test_distill_all_other_columns_masked(spmv, dtype, rows):
    """By the lowest value: they share the remainder's gradient evenly.  By -inf: the loss is +inf (the
    teacher has mass where the student cannot), the entries' gradient stays, the others' is 0."""
    vocab, k = 24, 20
    ids = torch.arange(k, dtype=torch.int32).repeat(rows, 1) + 4
    teacher = torch.linspace(0, 2, k).repeat(rows, 1)
    lse = (torch.logsumexp(teacher.double(), 1) + 0.1).float()
    rest = 1 - math.exp(-0.1)
    args = (ids.cuda(), teacher.cuda())
    for low in (torch.finfo(dtype).min, -math.inf):
        z = torch.linspace(-1, 1, vocab).repeat(rows, 1)
        z[:, :4] = low
        z = z.to(dtype).cuda()
        loss, dz = spmv.distill_loss_grad(z, *args, teacher_lse=lse.cuda())
        res = spmv.distill_loss(z, *args, teacher_lse=lse.cuda())
        for got_loss, got in ((loss, dz), (res.loss, res.grad())):
            got = f64(got)
            want = ref.distill_grad(f64(z[0]), ids[0].numpy(), f64(teacher[0]), float(lse[0]))
            assert np.abs(got - want).max() <= 1e-5 + H[dtype] * np.abs(want).max()
            if low == -math.inf:
                assert torch.isinf(got_loss).all() and not got[:, :4].any()
            else:  # the remainder to float rounding of lse, then the output's
                assert np.abs(got[:, :4] + rest / 4).max() <= 1e-5 + H[dtype] * rest


# --------------------------------------------------------------------------- #
# streams, graphs, errors
# --------------------------------------------------------------------------- #


def test_given_stream_and_graph(spmv):
    g = gen(8)
    z = torch.randn(16, 5000, generator=g).cuda()
    x = torch.randn(3000, 64, generator=g).cuda()  # (a plan of several CTAs, two kernels)
    ids, teacher = (t.cuda() for t in some_target(16, 5000, 10, g))
    torch.cuda.synchronize()

    def step(stream=None):
        top = spmv.topk_rows(x, 2, weights="selected", stream=stream)
        plan = spmv.RoutePlan(top.ids, 64, align=8, stream=stream)
        xs = plan.dispatch(x, stream=stream)
        y = plan.combine(xs, top.weights, stream=stream)
        dys, dw = plan.combine_grad(x, xs, top.weights, stream=stream)
        loss, dz = spmv.distill_loss_grad(z, ids, teacher, stream=stream)
        return [top.ids, xs, y, dys, dw, top.grad(dw, stream=stream), loss, dz]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in got:
        t.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals_on_the_gpu(spmv):
    z = torch.zeros(4, 100, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    t = torch.zeros(4, 2, device="cuda")
    with pytest.raises(spmv.SpmvError):  # host memory
        spmv.distill_loss(z.cpu(), ids, t)
    with pytest.raises(spmv.SpmvError):
        spmv.topk_rows(z.cpu(), 2)
    with pytest.raises(spmv.SpmvError):  # dz over part of z
        buf = torch.zeros(500, device="cuda")
        spmv.distill_loss_grad(buf[:400].view(4, 100), ids, t, out=buf[4:404].view(4, 100))
    plan = spmv.RoutePlan(ids, 3)
    with pytest.raises(spmv.SpmvError):
        plan.dispatch(z, out=torch.zeros(plan.rows, 100))  # host memory
    with pytest.raises(ValueError):
        plan.combine(z[:3])
    with pytest.raises(TypeError):
        plan.combine_grad(z, torch.zeros(plan.rows, 100, device="cuda", dtype=torch.float16), t)
    with pytest.raises(ValueError):
        spmv.topk_rows(z, 2).grad(t)
    with pytest.raises(spmv.SpmvError):  # an address that is no multiple of the value size
        spmv._abi.spmv_topk_rows(3, 99, 2, z.data_ptr() + 2, 99, 1, 1.0, 0, ids, t)
