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
