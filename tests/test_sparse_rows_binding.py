"""What the Python objects of the sparse-row operators hand to the library: recorded by a stand-in for
it, on host tensors (nothing is computed)."""
import copy
import os
import pickle
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Recorder:
    """Stands in for the library: sizes are the library's, every other call is noted and succeeds."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        if name in ("spmv_route_rows", "spmv_route_workspace"):
            return getattr(self.lib, name)

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def rows(monkeypatch):
    import __graft_entry__

    __graft_entry__._build_module().build()
    from sparse_matrix_vector_csr_gb300 import sparse_rows

    monkeypatch.setattr(sparse_rows, "lib", Recorder(sparse_rows.lib))
    return sparse_rows


def plan_pointers(rows, plan):
    """(slots, sources) that dispatch, combine and combine_grad pass on, one pair a call"""
    x, ys, w = torch.zeros(6, 8), torch.zeros(plan.rows, 8), torch.zeros(6, 2)
    rows.lib.calls.clear()
    plan.dispatch(x), plan.combine(ys, w), plan.dispatch_grad(ys), plan.combine_grad(x, ys, w)
    return [(a[4], a[5] if "combine" not in n or "grad" in n else None) for n, a in rows.lib.calls]


@pytest.mark.parametrize("change", ["none", "deepcopy", "pickle", "assigned"])
def test_a_plan_passes_the_tensors_it_has(rows, change):
    plan = rows.RoutePlan(torch.zeros(6, 2, dtype=torch.int32), 4, align=2)
    kept = [plan.slots, plan.sources]  # (so that no other tensor gets their memory)
    if change == "deepcopy":
        plan = copy.deepcopy(plan)
    elif change == "pickle":
        plan = pickle.loads(pickle.dumps(plan))
    elif change == "assigned":
        plan.slots, plan.sources = plan.slots.clone(), plan.sources.clone()
    slots, sources = plan.slots.data_ptr(), plan.sources.data_ptr()
    if change != "none":
        assert slots != kept[0].data_ptr() and sources != kept[1].data_ptr()
    assert plan_pointers(rows, plan) == [(slots, sources), (slots, None), (slots, None), (slots, sources)]


@pytest.mark.parametrize("name,value,error", [
    ("slots", torch.zeros(5, 2, dtype=torch.int32), ValueError), ("slots", torch.zeros(6, 2, dtype=torch.int64), TypeError),
    ("sources", torch.zeros(3, dtype=torch.int32), ValueError), ("slots", torch.zeros(2, 6, dtype=torch.int32).t(), ValueError)])
def test_a_plan_refuses_other_tensors_in_its_place(rows, name, value, error):
    plan = rows.RoutePlan(torch.zeros(6, 2, dtype=torch.int32), 4, align=2)
    setattr(plan, name, value)
    with pytest.raises(error):
        plan.dispatch(torch.zeros(6, 8))
    with pytest.raises(error):
        plan.combine_grad(torch.zeros(6, 8), torch.zeros(plan.rows, 8), torch.zeros(6, 2))


STAR = """
import sys
sys.modules["torch"] = None  # as where it is not installed
from sparse_matrix_vector_csr_gb300 import *
assert SpmvMatrix and spmv_apply and "topk_rows" not in globals()
"""


def test_star_import_without_torch(rows):
    run = subprocess.run([sys.executable, "-c", STAR], cwd=ROOT, timeout=300, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-2000:]


def test_star_import_has_the_sparse_rows(rows):
    names = {}
    exec("from sparse_matrix_vector_csr_gb300 import *", names)
    assert all(n in names for n in ("topk_rows", "RoutePlan", "distill_loss", "SpmvMatrix", "spmv_apply"))


def test_gradient_of_combine_refuses_more_ctas_than_a_grid_has():
    import numpy as np
    import sparse_matrix_vector_csr_gb300 as spmv

    h, m = np.zeros(8, np.float32), (1 << 31) - 1
    for tokens, rows, status in ((m, 1, -5), (m - 10, 640, -5), (m - 10, 320, -1)):  # (-1: host memory)
        with pytest.raises(spmv.SpmvError) as e:
            spmv.spmv_route_combine_grad(tokens, 1, rows, 0, h, h, h, None, 0, None, 0, None, 0, h, 1, stream=0)
        assert e.value.status == status, (tokens, rows, str(e.value))
