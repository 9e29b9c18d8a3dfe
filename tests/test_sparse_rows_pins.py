"""The 64-bit statements of the sparse-row operators pinned: hand-made rows, gradients against
central differences; and refusals that come before any CUDA call."""
import numpy as np
import pytest

from oracle import sparse_rows as ref


def differences(f, x, eps=1e-5):
    g = np.zeros(len(x))
    for i in range(len(x)):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = (f(a) - f(b)) / (2 * eps)
    return g


def test_topk_row_ties_masks_and_nan():
    ids, vals = ref.topk_row([1.0, 3.0, 3.0, -np.inf, 2.0], 3)
    assert ids.tolist() == [1, 2, 4] and vals.tolist() == [3.0, 3.0, 2.0]
    ids, vals = ref.topk_row([-np.inf, -5.0, -np.inf], 2)
    assert ids.tolist() == [1, -1] and vals.tolist() == [-5.0, -np.inf]
    assert ref.topk_row([0.0, np.inf, np.nan], 2)[0].tolist() == [2, 1]
    assert ref.topk_row([-0.0, 0.0], 2)[0].tolist() == [0, 1]


@pytest.mark.parametrize("weighting", ["selected", "row"])
@pytest.mark.parametrize("tau", [1.0, 0.5])
def test_weights_gradient_is_the_difference(weighting, tau):
    rng = np.random.default_rng(5)
    x, k = rng.normal(size=9) * 2, 4
    dw = rng.normal(size=k)
    ids, vals = ref.topk_row(x, k)
    w = ref.top_weights(x, ids, vals, weighting, tau)

    def f(v):
        i, vv = ref.topk_row(v, k)
        assert i.tolist() == ids.tolist()
        return float(dw @ ref.top_weights(v, i, vv, weighting, tau))

    # error of a central difference: eps^2 times a third derivative of order 1 / tau^3, and rounding / eps
    np.testing.assert_allclose(ref.top_weights_grad(x, ids, w, dw, weighting, tau), differences(f, x), atol=1e-8)


def test_route_plan_by_hand():
    offsets, slots, sources = ref.route_plan([[1, 0], [1, -1], [2, 1]], 4, 2, 12)
    assert offsets.tolist() == [0, 2, 6, 8, 8]
    assert slots.tolist() == [[2, 0], [3, -1], [6, 4]]
    assert sources.tolist() == [1, -1, 0, 2, 5, -1, 4, -1, -1, -1, -1, -1]


def test_route_products_are_transposes():
    rng = np.random.default_rng(6)
    ids = rng.integers(-1, 5, (7, 3))
    rows = 21 + 5 * 3
    _, slots, _ = ref.route_plan(ids, 5, 4, rows)
    x, ys, w = rng.normal(size=(7, 6)), rng.normal(size=(rows, 6)), rng.normal(size=(7, 3))
    np.testing.assert_allclose((ref.dispatch(x, slots, rows) * ys).sum(), (x * ref.combine(ys, slots, None)).sum())
    dy = rng.normal(size=(7, 6))
    dys, dw = ref.combine_grad(dy, ys, slots, w)
    base = (ref.combine(ys, slots, w) * dy).sum()
    np.testing.assert_allclose((dys * ys).sum(), base)  # linear in ys and in w
    np.testing.assert_allclose((dw * w).sum(), base)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_distill_gradient_is_the_difference(tail, tau):
    rng = np.random.default_rng(7)
    z, ids, t = rng.normal(size=11) * 2, np.array([4, -1, 0, 9]), rng.normal(size=4) * 2
    norm = ref.lse(t[[0, 2, 3]] / tau) + 0.2 if tail else None
    g = ref.distill_grad(z, ids, t, norm, tau)
    np.testing.assert_allclose(g, differences(lambda v: ref.distill_loss(v, ids, t, norm, tau), z), atol=1e-8)
    np.testing.assert_allclose(g.sum(), 0.0, atol=1e-12)  # a constant added to z changes nothing


def test_distill_is_zero_where_student_equals_teacher_and_without_target():
    z = np.array([1.0, 2.0, -1.0, 0.5])
    assert abs(ref.distill_loss(z, [1, 3], z[[1, 3]], ref.lse(z))) < 1e-12
    assert ref.distill_loss(z, [-1, 7], [0.0, 0.0]) == 0.0
    assert not ref.distill_grad(np.full(4, np.nan), [-1, -1], [0.0, 0.0]).any()


# --------------------------------------------------------------------------- #
# refusals before any CUDA call (host arrays stand in for device ones, nothing is read)
# --------------------------------------------------------------------------- #


@pytest.fixture(scope="module")
def spmv():
    import __graft_entry__

    __graft_entry__._build_module().build()
    import sparse_matrix_vector_csr_gb300 as spmv

    return spmv


D = np.zeros(64, np.float32)


def refused(spmv, status, fn, *args):
    with pytest.raises(spmv.SpmvError) as e:
        fn(*args, stream=0)
    assert e.value.status == status, str(e.value)


@pytest.mark.parametrize("change", [
    {"rows": -1}, {"rows": 1 << 31}, {"n": 1 << 31}, {"k": 0}, {"k": 9}, {"k": 257, "n": 1000, "ldx": 1000}, {"ldx": 7}, {"dtype": 0}, {"dtype": 4},
    {"temperature": 0.0}, {"temperature": float("nan")}, {"temperature": -1.0}, {"weighting": 3}, {"x": None}, {"ids": None},
    {"weighting": 1, "weights": None}])
def test_topk_rows_refusals(spmv, change):
    a = {"rows": 2, "n": 8, "k": 2, "x": D, "ldx": 8, "dtype": 1, "temperature": 1.0, "weighting": 0, "ids": D,
         "vals": D, "weights": D, "lse": D, **change}
    refused(spmv, -1, spmv.spmv_topk_rows, *a.values())


@pytest.mark.parametrize("change", [{"weighting": 0}, {"weighting": 3}, {"k": 0}, {"lddx": 7}, {"dx": None}, {"dtype": 0},
                                    {"temperature": 0.0}, {"dweights": None}])
def test_topk_rows_grad_refusals(spmv, change):
    a = {"rows": 2, "n": 8, "k": 2, "ids": D, "weights": D, "dweights": D, "weighting": 1, "temperature": 1.0,
         "x": None, "ldx": 0, "lse": None, "dx": D, "lddx": 8, "dtype": 1, **change}
    refused(spmv, -1, spmv.spmv_topk_rows_grad, *a.values())


def test_route_sizes(spmv):
    assert spmv.spmv_route_rows(4, 8, 128, 1) == 32
    assert spmv.spmv_route_rows(4, 8, 128, 16) == 32 * 16
    assert spmv.spmv_route_rows(1000, 2, 7, 16) == (2000 + 7 * 15) // 16 * 16
    assert spmv.spmv_route_rows(0, 8, 128, 16) == 0
    assert spmv.spmv_route_workspace(4, 8, 128) == 0
    assert spmv.spmv_route_workspace(1 << 20, 8, 128) > 0
    for args, status in (((-1, 1, 4, 1), -1), ((4, 0, 4, 1), -1), ((4, 1, 0, 1), -1), ((4, 1, 4097, 1), -1),
                         ((4, 1, 4, 0), -1), ((4, 1, 4, 65537), -1), ((1 << 30, 2, 4, 1), -5),
                         ((1 << 29, 2, 4096, 65536), None), (((1 << 31) - 1, 1, 4096, 65536), -5)):
        if status is None:
            assert spmv.spmv_route_rows(*args) < 1 << 31
            continue
        with pytest.raises(spmv.SpmvError) as e:
            spmv.spmv_route_rows(*args)
        assert e.value.status == status, args


def test_route_refusals(spmv):
    refused(spmv, -1, spmv.spmv_route_plan, 4, 0, 8, 1, D, D, D, D, None, 0)
    refused(spmv, -1, spmv.spmv_route_plan, 1 << 20, 8, 8, 1, D, D, D, D, D, 16)  # workspace too small
    refused(spmv, -1, spmv.spmv_route_plan, 4, 2, 8, 1, D, None, D, D, None, 0)
    refused(spmv, -1, spmv.spmv_route_dispatch, 4, 2, 8, 16, D, D, D, 15, D, 16, 1)  # ldx < d
    refused(spmv, -1, spmv.spmv_route_dispatch, 4, 2, 8, 16, D, D, D, 16, D, 16, 0)  # float64
    refused(spmv, -1, spmv.spmv_route_combine, 4, 2, 8, 16, D, D, D, 16, None, 16, 1)
    refused(spmv, -1, spmv.spmv_route_combine, 4, 2, -8, 16, D, D, D, 16, D, 16, 1)
    refused(spmv, -1, spmv.spmv_route_combine_grad, 4, 2, 8, 16, D, D, None, D, 16, D, 16, D, 16, D, 1)
    refused(spmv, -5, spmv.spmv_route_combine, 1 << 30, 4, 8, 16, D, D, D, 16, D, 16, 1)


@pytest.mark.parametrize("change, status", [
    ({"rows": -1}, -1), ({"vocab": 0, "ldz": 0}, -1), ({"vocab": (1 << 22) + 1, "ldz": 1 << 23}, -5), ({"ldz": 7}, -1), ({"k": 0}, -1),
    ({"k": 513}, -1), ({"dtype": 0}, -1), ({"teacher_dtype": 7}, -1), ({"temperature": 0.0}, -1),
    ({"temperature": float("inf")}, -1), ({"z": None}, -1), ({"ids": None}, -1), ({"teacher": None}, -1), ({"loss": None}, -1)])
def test_distill_refusals(spmv, change, status):
    a = {"rows": 2, "vocab": 8, "k": 2, "z": D, "ldz": 8, "dtype": 1, "ids": D, "teacher": D, "teacher_dtype": 1,
         "teacher_lse": None, "temperature": 1.0, "loss": D, **change}
    refused(spmv, status, spmv.spmv_distill_loss, *a.values())
    refused(spmv, status, spmv.spmv_distill_loss_grad, *a.values(), 1.0, None, D, max(8, a["ldz"]))


def test_distill_grad_refusals(spmv):
    a = [2, 8, 2, D, 8, 1, D, D, 1, None, 1.0]
    refused(spmv, -1, spmv.spmv_distill_grad, *a, D, float("nan"), None, D, 8)  # scale
    refused(spmv, -1, spmv.spmv_distill_grad, *a, D, 1.0, None, D, 7)  # lddz
    refused(spmv, -1, spmv.spmv_distill_grad, *a, None, 1.0, None, D, 8)  # stats
    # no rows: nothing to do, nothing read
    spmv.spmv_distill_loss(0, 8, 2, None, 8, 1, None, None, 1, None, 1.0, None, None, 0)
    spmv.spmv_topk_rows(0, 8, 2, None, 8, 1, 1.0, 0, None, None, None, None, 0)


def test_python_argument_checks(spmv):
    import torch

    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        spmv.topk_rows(x.double(), 2)
    with pytest.raises(ValueError):
        spmv.topk_rows(x, 9)
    with pytest.raises(ValueError):
        spmv.topk_rows(x.t(), 2)
    with pytest.raises(KeyError):
        spmv.topk_rows(x, 2, weights="all")
    with pytest.raises(TypeError):
        spmv.RoutePlan(torch.zeros(4, 2), 8)
    with pytest.raises(TypeError):
        spmv.distill_loss(x, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        spmv.distill_loss(x, torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2))
    with pytest.raises(ValueError):
        spmv.distill_loss(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 3))
    with pytest.raises(ValueError):
        spmv.distill_loss(torch.zeros(1, 8).expand(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
