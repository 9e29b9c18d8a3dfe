"""The sparse-row operators at the edges of their ranges, on the GPU: sizes at a limit, masks by the type's
lowest value, offsets far from 0, infinities, states that change between two calls.

E, H, TINY and SUM are the units of tests/test_gpu_sparse_rows.py: half a unit of a float, of the output's
type, its smallest values, and the relative error of a sum of hardware exponentials.
"""
import copy
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import sparse_rows as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E = 2.0 ** -24
H = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-37}
SUM = 2e-5
ALL = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def spmv():
    import __graft_entry__

    __graft_entry__._build_module().build()
    import sparse_matrix_vector_csr_gb300 as spmv

    return spmv


def f64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    return torch.Generator().manual_seed(seed)


# --------------------------------------------------------------------------- #
# rows sorted by expert
# --------------------------------------------------------------------------- #


PLAN = """
import sys
import torch
import sparse_matrix_vector_csr_gb300 as spmv
from oracle import sparse_rows as ref
tokens, k, experts = map(int, sys.argv[1:])
ids = torch.randint(-1, experts, (tokens, k), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
plan = spmv.RoutePlan(ids.cuda(), experts)
want = ref.route_plan(ids.numpy(), experts, 1, plan.rows)
assert all((a.cpu().numpy() == b).all() for a, b in zip((plan.offsets, plan.slots, plan.sources), want))
"""


@pytest.mark.parametrize("tokens,k,experts", [(4, 8, 4096), (4, 8, 4091), (8, 8, 3072), (16, 8, 2048), (40, 5, 1228),
                                              (1000, 4, 682), (1000, 4, 1228)])
def test_route_plan_at_the_shared_memory_limit(spmv, tokens, k, experts):
    """The plan's shared memory ends at or just below 48 KB: the first call of a process, since one that
    needs more leaves the kernel with a larger limit."""
    run = subprocess.run([sys.executable, "-c", PLAN, str(tokens), str(k), str(experts)], cwd=ROOT, timeout=300,
                         capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-2000:]


def test_route_plan_of_nearly_2_to_the_31_entries(spmv):
    """One expert has them all, and its segment's end, rounded up to whole tiles, passes 2^31 on the way."""
    m = 2 ** 31 - 2  # a multiple of 3; m + 2 is 2^31
    plan = spmv.RoutePlan(torch.zeros(m, 1, dtype=torch.int32, device="cuda"), 1, align=3)
    assert plan.rows == m and plan.offsets.tolist() == [0, m]
    for a in range(0, m, 1 << 28):
        want = torch.arange(a, min(m, a + (1 << 28)), dtype=torch.int32, device="cuda")
        assert torch.equal(plan.slots[a:a + len(want), 0], want) and torch.equal(plan.sources[a:a + len(want)], want)


# --------------------------------------------------------------------------- #
# the k largest entries of each row
# --------------------------------------------------------------------------- #


def check_weights_grad(spmv, x, k, weighting, tau, seed):
    """dx against the softmax's Jacobian in 64 bits, from differences to the row's maximum."""
    rows, n = x.shape
    top = spmv.topk_rows(x, k, temperature=tau, weights=weighting)
    dw = torch.randn(rows, k, generator=gen(seed)).cuda()
    got, ids, d = f64(top.grad(dw)), top.ids.cpu().numpy(), f64(dw)
    for r, row in enumerate(f64(x)):
        cols, dj = ids[r][ids[r] >= 0], d[r][ids[r] >= 0]
        assert len(cols) == min(k, int((row > -np.inf).sum()))
        share = np.zeros(n)
        over = cols if weighting == "selected" else np.flatnonzero(row > -np.inf)
        if len(cols):
            share[over] = np.exp((row[over] - row.max()) / tau)
            share /= share.sum()
        dot = (share[cols] * dj).sum()
        want = -share * dot
        want[cols] += share[cols] * dj
        size = share * np.abs(share[cols] * dj).sum()
        size[cols] += np.abs(share[cols] * dj)
        # an exponential's argument is a difference, rounded relative to itself; weights and sums: 2 SUM each
        np.testing.assert_array_less(np.abs(got[r] - want / tau),
                                     4 * SUM * size / tau + H[x.dtype] * np.abs(want) / tau + TINY[x.dtype])


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("weighting", ["row", "selected"])
@pytest.mark.parametrize("tau", [0.7, 1.0, 2.0])
@pytest.mark.parametrize("n,k", [(40, 3), (300, 16), (512, 5), (40, 20), (700, 3), (5000, 40)])
def test_weights_gradient_of_lowest_values_and_far_from_0(spmv, dtype, weighting, tau, n, k):
    low = torch.finfo(dtype).min
    x = torch.randn(8, n, generator=gen(n)) * 2
    x[0] = low                    # wholly masked by the lowest value: n equal shares
    x[1] = low
    x[1, n // 3] = 1.0            # one column left
    x[2, n // 2:] = low
    x[3] += 1e4                   # ordinary differences, far from 0
    x[4] -= 1e4
    x[5, ::2] = -math.inf
    x[5, 1::2] = low              # both masks
    x[6] = -math.inf
    x[7] = -3e4 if dtype == torch.float16 else -1e30
    check_weights_grad(spmv, x.to(dtype).cuda(), k, weighting, tau, n + k)


@pytest.mark.parametrize("weighting", [1, 2])
@pytest.mark.parametrize("n,k", [(40, 6), (40, 20), (700, 6)])
def test_weights_gradient_leaves_out_columns_outside(spmv, weighting, n, k):
    """An entry whose column is n or more is no entry, as one of -1 is none: its weight enters nothing."""
    g = gen(n)
    x = torch.randn(3, n, generator=g).cuda()
    ids, lse = (torch.empty(s, dtype=t, device="cuda") for s, t in (((3, k), torch.int32), ((3,), torch.float32)))
    w, dw = torch.empty(3, k, device="cuda"), torch.randn(3, k, generator=g).cuda()
    spmv.spmv_topk_rows(3, n, k, x, n, 1, 1.0, weighting, ids, None, w, lse)
    got = []
    for outside in (-1, n, 2 ** 31 - 1):
        ids[:, 2], ids[1, 4] = outside, outside
        dx = torch.full_like(x, math.nan)
        spmv.spmv_topk_rows_grad(3, n, k, ids, w, dw, weighting, 1.0, x, n, lse, dx, n, 1)
        got.append(dx)
    assert torch.isfinite(got[0]).all() and torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("n,k", [(40, 3), (512, 16), (40, 20), (600, 3), (3000, 8), (150000, 8)])
def test_log_sum_of_a_row_with_infinity(spmv, dtype, n, k):
    """The sum of exponentials is +inf, and so is its log; with a NaN beside it, NaN."""
    x = torch.randn(6, n, generator=gen(n))
    x[0, n // 2] = math.inf
    x[1] = math.inf
    x[2, [1, n - 1]] = math.inf
    x[2, 3:n - 3] = -math.inf
    x[3, 5], x[3, n - 2] = math.inf, math.nan
    x[4, n - 1] = math.nan
    x = x.to(dtype).cuda()
    for tau in (0.5, 1.0, 3.0):
        top = spmv.topk_rows(x, k, temperature=tau, lse=True)
        lse = f64(top.lse)
        assert (lse[:3] == math.inf).all() and np.isnan(lse[3:5]).all() and np.isfinite(lse[5])
        assert top.ids[:3, 0].tolist() == [n // 2, 0, 1]
        with np.errstate(invalid="ignore"):
            want = [ref.lse(row / tau) for row in f64(x)]
        np.testing.assert_array_equal(lse[:5], want[:5])


def order_keys(x):
    """(value's order, lowest column first) as one int64 a value; -inf below everything."""
    f = x.float() + 0.0
    bits = f.view(torch.int32)
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64)
    bits = torch.where(torch.isnan(f), torch.full_like(bits, 0x7F800001), bits)
    return bits * (1 << 32) + (x.shape[1] - 1 - torch.arange(x.shape[1], device=x.device))


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,n,k", [(620, 131077, 64), (620, 131077, 200), (613, 300001, 17)])
def test_topk_of_many_long_rows(spmv, dtype, rows, n, k):
    """Rows so long that several pieces share a maximum, in batches as a teacher's logits come in."""
    x = torch.randn(rows, n, generator=torch.Generator(device="cuda").manual_seed(n + k), device="cuda").mul_(2).to(dtype)
    size = x.element_size()
    per_vec, threads = 16 // size, 256 if k <= 128 else 512
    pieces = -(-(-(-(n + per_vec - 1) // per_vec)) // (threads * (16 // per_vec)))
    per = 1
    while -(-pieces // per) > 15:
        per *= 2
    assert per > 1
    for r in range(0, 12):  # the largest entries at a slot's last piece, at the row's ends, behind one another
        head = (x[r].data_ptr() % 16) // size
        lo = 1 if head else 0
        at = []
        for j in range(k):
            t, s = (37 * j + r) % threads, j % (pieces // per)
            piece = s * per + (per - 1 if r % 2 == 0 else j % per)
            vec = lo + t + (piece * (16 // per_vec) + j % (16 // per_vec)) * threads
            at.append(vec * per_vec - head + (j % per_vec))
        if r in (1, 2):
            at = [0, n - 1, 1, n - 2] + at
        if r == 3:
            at = list(range(n - k, n))
        if r == 4:
            at = list(range(k))
        at = torch.tensor([c for c in at if 0 <= c < n])
        x[r, at] = (20 + torch.rand(len(at), generator=gen(r)) * 8).to(dtype).cuda()
    x[12] = 1.0
    x[13] = torch.arange(n, device="cuda").div(n)
    x[14, :-3] = -math.inf
    x[15, n // 2], x[15, n - 1] = math.nan, math.nan
    x[16] = torch.finfo(dtype).min
    top = spmv.topk_rows(x, k, lse=True)
    for a in range(0, rows, 100):
        part = x[a:a + 100]
        cols = n - 1 - (order_keys(part).topk(k, dim=1).values & 0xFFFFFFFF)
        vals = part.float().gather(1, cols)
        cols = torch.where(vals == -math.inf, torch.full_like(cols, -1), cols)
        assert torch.equal(top.ids[a:a + 100].long(), cols)
        assert torch.equal(torch.nan_to_num(top.vals[a:a + 100], nan=7.0), torch.nan_to_num(vals, nan=7.0))
        norm = torch.logsumexp(part.double(), 1)
        near = (top.lse[a:a + 100].double() - norm).abs() <= SUM + 4 * E * norm.abs()
        assert (near | torch.isnan(norm)).all() and torch.equal(torch.isnan(norm), torch.isnan(top.lse[a:a + 100]))
    for r in (0, 3, 12, 14, 15, 100):
        ids, vals = ref.topk_row(f64(x[r]), k)
        assert np.array_equal(top.ids[r].cpu().numpy(), ids) and np.array_equal(f64(top.vals[r]), vals, equal_nan=True)


# --------------------------------------------------------------------------- #
# distillation
# --------------------------------------------------------------------------- #


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows", [3, 1300])
@pytest.mark.parametrize("vocab", [24, 9000])
@pytest.mark.parametrize("tau", [0.5, 1.0, 2.0])
def test_distill_remainder_where_the_others_are_lowest(spmv, dtype, rows, vocab, tau):
    """The student has the teacher's logits and every other column masked by the type's lowest value.  A
    remainder that is the rounding of lse counts as 0, as it does beside a mask of -inf: no loss, no gradient.
    A real one meets the logits that are there, and overflows no sooner than the loss itself."""
    k = 20
    ids = torch.arange(k, dtype=torch.int32).repeat(rows, 1) + 2
    low = torch.finfo(dtype).min
    z = torch.full((rows, vocab), low)
    z[:, 2:2 + k] = torch.linspace(0, 2, k).to(dtype).float()
    z = z.to(dtype).cuda()
    teacher = z[:, 2:2 + k].float()
    args = (z, ids.cuda(), teacher.contiguous())
    full = torch.logsumexp(teacher.double() / tau, 1)
    for extra in (2e-6, 0.1):
        lse = (full + extra).float()
        loss, dz = spmv.distill_loss_grad(*args, teacher_lse=lse, temperature=tau)
        res = spmv.distill_loss(*args, teacher_lse=lse, temperature=tau)
        rest = -math.expm1(-extra)
        for got_loss, got in ((loss, dz), (res.loss, res.grad())):
            if extra < 1e-5:
                # p and q agree to the rounding of lse (2^-23 of it, and 2e-6), the loss is of their first order
                assert got_loss.abs().max() <= 1e-5 + SUM
                assert not got[:, :2].any() and not got[:, 2 + k:].any()
                assert got.float().abs().max() <= (1e-5 + SUM) / tau
                continue
            # rest, from 32 bits, to 1e-5 of 0.1
            want = rest * (2.0 - float(low)) / tau
            got = f64(got)
            assert np.abs(f64(got_loss) / want - 1).max() <= 1e-3
            others = np.delete(got, np.arange(2, 2 + k), 1)
            size = rest / (vocab - k) / tau
            assert np.abs(others + size).max() <= (1e-3 + H[dtype]) * size + TINY[dtype]


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,vocab", [(3, 40), (3, 9000), (1300, 40)])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_rows_whose_mask_leaves_nothing(spmv, dtype, rows, vocab, tail):
    """No softmax, so NaN where there is a target, 0 where there is none; the rows beside them as ever."""
    z = (torch.randn(rows, vocab, generator=gen(vocab)) * 2).to(dtype).cuda()
    ids = torch.arange(5, dtype=torch.int32).repeat(rows, 1).cuda() * 7
    teacher = torch.randn(rows, 5, generator=gen(rows)).cuda()
    lse = torch.logsumexp(teacher, 1) + 0.2 if tail else None
    plain = spmv.distill_loss_grad(z, ids, teacher, teacher_lse=lse)
    z[0], z[1] = -math.inf, -math.inf
    ids[1] = -1
    loss, dz = spmv.distill_loss_grad(z, ids, teacher, teacher_lse=lse)
    res = spmv.distill_loss(z, ids, teacher, teacher_lse=lse)
    for got_loss, got in ((loss, dz), (res.loss, res.grad())):
        assert torch.isnan(got_loss[0]) and torch.isnan(got[0, ids[0].long()]).all()
        assert got_loss[1] == 0 and not got[1].any()
    assert torch.equal(loss[2:], plain[0][2:]) and torch.equal(dz[2:], plain[1][2:])


# --------------------------------------------------------------------------- #
# states between two calls
# --------------------------------------------------------------------------- #


def test_weights_gradient_is_that_of_the_weights_given(spmv):
    """Other tensors in the attributes' place (scaled weights, dropped entries) change nothing."""
    x = torch.randn(30, 64, generator=gen(5)).cuda()
    dw = torch.randn(30, 4, generator=gen(6)).cuda()
    for weighting in ("selected", "row"):
        top = spmv.topk_rows(x, 4, weights=weighting)
        want = top.grad(dw)
        top.weights, top.ids, top.lse = top.weights * 2.5, top.ids[:2], None
        assert torch.equal(top.grad(dw), want)
        assert torch.equal(copy.deepcopy(top).grad(dw), want)


def test_distill_gradient_is_that_of_the_loss_given(spmv):
    z = torch.randn(30, 64, generator=gen(5)).cuda()
    ids = torch.arange(4, dtype=torch.int32, device="cuda").repeat(30, 1)
    teacher = torch.randn(30, 4, generator=gen(6)).cuda()
    res = spmv.distill_loss(z, ids, teacher)
    want = res.grad()
    res.stats, res.loss = torch.zeros_like(res.stats), None
    assert torch.equal(res.grad(), want)
    assert torch.equal(copy.deepcopy(res).grad(), want)
