"""The feed-forward block where its kernels change shape and where values leave their range, against its 64-bit
statement (oracle/token_rows.py).  The helpers and how their tolerances are derived: test_gpu_feed_forward.py."""
import math
import threading

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


@pytest.mark.parametrize("dtype", ALL)
def test_first_call_of_a_host_thread(spmv, dtype):
    """a host thread that has made no CUDA call yet: the library's is the first"""
    from sparse_matrix_vector_csr_gb300._abi import _check, lib

    g, code = gen(2), {torch.float32: 1, torch.float16: 2, torch.bfloat16: 3}[dtype]
    x, dy = torch.randn(40, 64, generator=g).to(dtype).cuda(), torch.randn(40, 64, generator=g).to(dtype).cuda()
    ws = weights(None, 64, 72, dtype, g)
    want = spmv.feed_forward(x, *ws, keep=True)
    want_dx = want.grad(dy)[0]
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    sizes = [spmv.spmv_feed_forward_workspace(40, 64, 72, 1, code, gradient) for gradient in (0, 1)]
    spaces = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    call = (40, 64, 72, 1, None, x.data_ptr(), 64, ws[0].data_ptr(), ws[1].data_ptr(), 64, 0, ws[2].data_ptr(), 72, 0, 0)
    forward = (*call, None, None, 72, y.data_ptr(), 64, code, spaces[0].data_ptr(), sizes[0], None)
    back = (*call, want.gate.data_ptr(), want.up.data_ptr(), want.gate.stride(0), dy.data_ptr(), 64, dx.data_ptr(), 64, None, None, None, code,
            spaces[1].data_ptr(), sizes[1], None)
    torch.cuda.synchronize()
    failed = []

    def work(entry, args):
        try:
            _check(entry(*args))
        except spmv.SpmvError as e:
            failed.append(str(e))

    for entry, args in ((lib.spmv_feed_forward, forward), (lib.spmv_feed_forward_grad, back)):
        t = threading.Thread(target=work, args=(entry, args))
        t.start()
        t.join()
    assert not failed, failed
    torch.cuda.synchronize()
    assert torch.equal(y, want.y) and torch.equal(dx, want_dx)


def test_calls_of_two_threads(spmv):
    """blocks of few and of many experts, which share kernels and need different amounts of shared memory, from two
    host threads at once (a call's arguments made beforehand: the threads meet inside the library)"""
    g = gen(1)
    sets = []
    for experts, rows in ((2, 6), (4096, 300)):
        plan, x, _, _ = routed(spmv, rows, 1, experts, 1, 64, torch.bfloat16, g, dropped=0.0)
        ws, y, stream = weights(experts, 64, 72, torch.bfloat16, g), torch.zeros_like(x), torch.cuda.Stream()
        n = spmv.spmv_feed_forward_workspace(rows, 64, 72, experts, 3)
        space = torch.empty(n, dtype=torch.uint8, device="cuda")
        args = (rows, 64, 72, experts, plan.offsets.data_ptr(), x.data_ptr(), 64, ws[0].data_ptr(), ws[1].data_ptr(), 64, 64 * 72,
                ws[2].data_ptr(), 72, 64 * 72, 0, None, None, 72, y.data_ptr(), 64, 3, space.data_ptr(), n, stream.cuda_stream)
        sets.append((args, plan.feed_forward(x, *ws).y, y, stream, (plan, x, ws, space)))
    torch.cuda.synchronize()
    from sparse_matrix_vector_csr_gb300._abi import _check, lib

    refused = []

    def work(i):
        args, _, _, stream, _ = sets[i]
        for n in range(4000):
            try:
                _check(lib.spmv_feed_forward(*args))
            except spmv.SpmvError as e:
                refused.append((i, n, str(e)))
            if n % 200 == 0:
                stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, refused
    assert all(torch.equal(want, y) for _, want, y, _, _ in sets)


def activations(spmv, gates, act, dtype):
    """(act, act') of the gates as the block computes them: x is a unit row, up is 1, w_down the identity and dy 1, so that y and the
    gradients in the first columns of w_up and w_gate are single products with 1"""
    n = len(gates)
    x = torch.zeros(1, n, dtype=dtype, device="cuda")
    x[0, 0] = 1.0
    wg, wu = (torch.zeros(n, n, dtype=dtype, device="cuda") for _ in range(2))
    wg[:, 0], wu[:, 0] = gates.to(dtype).cuda(), 1.0
    res = spmv.feed_forward(x, wg, wu, torch.eye(n, dtype=dtype, device="cuda"), activation=act, keep=True)
    _, dwg, dwu, _ = res.grad(torch.ones_like(x))
    assert torch.equal(res.gate[0].cpu(), gates.to(dtype))
    return f64(res.y[0]), f64(dwu[:, 0]), f64(dwg[:, 0])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_float_activations(spmv, act):
    """act and act' of float rows to 32 bits relative to their value, over the whole range of the exponential.

    With E = 2^-23 and v the exponent (x, or gelu's 2 z): the exponential and the quotient, which is at least 1/2, are within 2 E (two
    units in the last place), 1 + e and the product add E / 2 each, so s and 1 - s are within 5 E and x s within 5.5 E.  gelu's 2 z is
    within 3 E of its value (two constants, four operations), which the exponential turns into 3 E |v|.  An exponential below
    2^-126 is within two of the smallest steps, 2^-148.
    """
    gates = torch.cat([torch.linspace(-110, 110, 441), torch.linspace(-12, 12, 389), torch.tensor([-1e-30, 0.0, 1e-30, 1e18, -1e18])])
    x = f64(gates)
    if act == "silu":
        v, dv = x, np.ones_like(x)
    else:
        v = 2 * np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)
        dv = 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * x * x)
    E, lost = 2.0 ** -23, 2.0 ** -148
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        e = np.exp(-np.abs(v))
        s, c = np.where(v < 0, e, 1) / (1 + e), np.where(v < 0, 1, e) / (1 + e)  # s and 1 - s, without a difference
        value, part = x * s, np.where(c * s == 0, 0.0, x * s * c * dv)
    slope = s + part
    off = 3 * E * np.abs(v) if act == "gelu_tanh" else 0 * v
    off = np.minimum(off, 1.0)  # (beyond it s is 0 or 1 and its error the smallest step's)
    y, by_up, by_gate = activations(spmv, gates, act, torch.float32)
    bound = (5.5 * E + off) * np.abs(value) + 2 * lost * (1 + np.abs(x))
    within_ = lambda got, want, b: np.argwhere(~(np.abs(got - want) <= b))[:5].ravel().tolist()  # noqa: E731
    assert not within_(y, value, bound), [(x[i], y[i], value[i]) for i in within_(y, value, bound)]
    assert np.array_equal(by_up, y)
    # s, x s (1 - s) and their sum; 5 E + E / 2 each, gelu's slope of 2 z 3 E, and roundings
    bound = (15 * E + 2 * off) * (s + np.abs(part)) + 4 * lost * (1 + np.abs(x)) * (1 + np.minimum(np.abs(dv), 1e3))
    assert not within_(by_gate, slope, bound), [(x[i], by_gate[i], slope[i]) for i in within_(by_gate, slope, bound)]
