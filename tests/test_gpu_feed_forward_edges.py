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


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows", [8, 9, 12, 16, 17])
@pytest.mark.parametrize("d,f", [(72, 200), (136, 1032), (9800, 40)])
def test_few_dense_rows(spmv, dtype, rows, d, f):
    """tiles of 8 and of 16 rows, w_down's of 32 columns and (d = 9800) of 64, and the first size beyond them"""
    g = gen(rows + d)
    x, dy = torch.randn(rows, d, generator=g).to(dtype).cuda(), torch.randn(rows, d, generator=g).to(dtype).cuda()
    ws = weights(None, d, f, dtype, g)
    check(spmv, x, ws, "silu", dy, [(0, rows)], lambda keep: spmv.feed_forward(x, *ws, keep=keep))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 8, 9, 16])
@pytest.mark.parametrize("d,f", [(72, 200), (9800, 40)])
def test_few_rows_keep_what_rounding_leaves(spmv, dtype, rows, d, f):
    """y of up to 16 rows with a bound that leaves no room for h's rounding: what that leaves out is rounded (H of it) and kept"""
    g = gen(rows + f)
    x, ws, half = torch.randn(rows, d, generator=g).to(dtype).cuda(), weights(None, d, f, dtype, g), H[dtype]
    w = [f64(t) for t in ws]
    y, sums = ref.feed_forward(f64(x), *w, "relu", unit=U, half=0.0, tiny=0.0)["y"]
    h = np.maximum(f64(x) @ w[0].T, 0) * (f64(x) @ w[1].T)
    kept = sums + (half * half * np.abs(h) + 2 * TINY[dtype]) @ np.abs(w[2]).T
    within(spmv.feed_forward(x, *ws, activation="relu").y, y, kept + half * (np.abs(y) + kept) + TINY[dtype], "y")


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("entries,experts,hot", [(200, 64, 0), (448, 64, 0), (500, 64, 150), (250, 64, 70), (30, 5, 0)])
@pytest.mark.parametrize("d,f", [(256, 72), (88, 264)])
def test_short_segments(spmv, dtype, entries, experts, hot, d, f):
    """segments of a few rows, in tiles of 8 (mean 4) and of 16 (mean 7 and 8); with one expert far beyond the mean"""
    g = gen(entries + d)
    ids = torch.randint(0, experts, (entries,), generator=g, dtype=torch.int32)
    ids[:hot] = 3
    plan = spmv.RoutePlan(ids[torch.randperm(entries, generator=g)][:, None].cuda(), experts)
    xs, dys = (plan.dispatch(torch.randn(entries, d, generator=g).to(dtype).cuda()) for _ in range(2))
    offsets = plan.offsets.tolist()
    ws = weights(experts, d, f, dtype, g)
    check(spmv, xs, ws, "gelu_tanh", dys, list(zip(offsets, offsets[1:])),
          lambda keep: plan.feed_forward(xs, *ws, activation="gelu_tanh", keep=keep))


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("entries,experts,d,f", [(3400, 48, 264, 280), (1500, 24, 1032, 1000), (3400, 48, 280, 512)])
def test_many_middling_segments(spmv, dtype, entries, experts, d, f):
    """tiles of 128 x 256 (gate and up: 2 x 128) by one CTA each: segments of about 70 rows, enough of them for 96 SMs"""
    g = gen(entries + d)
    plan, xs, dys, spans = routed(spmv, entries, 1, experts, 1, d, dtype, g)
    ws = weights(experts, d, f, dtype, g)
    check(spmv, xs, ws, "silu", dys, spans, lambda keep: plan.feed_forward(xs, *ws, keep=keep))


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,d,f", [(8200, 256, 256), (4200, 264, 280)])
def test_wide_weights_in_parts(spmv, dtype, rows, d, f):
    """the weights' gradients by pairs of CTAs and in parts of the rows at once"""
    g = gen(rows)
    x, dy = torch.randn(rows, d, generator=g).to(dtype).cuda(), torch.randn(rows, d, generator=g).to(dtype).cuda()
    ws = weights(None, d, f, dtype, g)
    check(spmv, x, ws, "relu", dy, [(0, rows)], lambda keep: spmv.feed_forward(x, *ws, activation="relu", keep=keep))


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,d,f", [(2, 2117, 2205), (16, 2117, 2205), (28, 1029, 2205), (32, 2117, 1061), (33, 1029, 1061),
                                      (1300, 301, 3561), (1300, 3561, 301)])
def test_long_sums_by_the_ordinary_units(spmv, dtype, rows, d, f):
    """odd sizes: tiles of 32 and of 128 rows, each tile's k shared by a cluster and (1300 rows) not, sums of more than 256 of k"""
    g = gen(rows + d)
    x, dy = torch.randn(rows, d, generator=g).to(dtype).cuda(), torch.randn(rows, d, generator=g).to(dtype).cuda()
    ws = weights(None, d, f, dtype, g)
    check(spmv, x, ws, "silu", dy, [(0, rows)], lambda keep: spmv.feed_forward(x, *ws, keep=keep))


@pytest.mark.parametrize("rows,d,f", [(2, 2117, 2205), (28, 2117, 2205), (1300, 301, 3561)])
def test_float_sums_do_not_grow_with_k(spmv, rows, d, f):
    """Sums of float products in parts of 256: n terms of the size t have a total whose rounding is at most 2^-23 times
    256 + n / 256 + 8 additions of sums of up to n t (and not n); against products in 64 bits."""
    g = gen(f)
    x = torch.rand(rows, d, generator=g).cuda() + 0.5  # (no cancelling: the rounding of the partial sums adds up)
    ws = [(torch.rand(w.shape, generator=g) + 0.5).cuda() / w.shape[-1] for w in weights(None, d, f, torch.float32, g)]
    res = spmv.feed_forward(x, *ws, activation="relu", keep=True)
    gate = x.double() @ ws[0].double().t()
    y = (res.gate.double() * res.up.double()) @ ws[2].double().t()
    for got, want, n in ((res.gate, gate, d), (res.y, y, f)):
        assert float(((got.double() - want).abs() / want).max()) <= 2.0 ** -23 * (256 + n / 256 + 8), n


def guarded(shape, dtype, shift=0, pad=0):
    """(a matrix of zeros, the NaN around it: all of the buffer)"""
    view = placed(torch.zeros(shape, dtype=dtype), shift, pad)
    return view, view._base if view._base is not None else view


def untouched(view, buf):
    inside = torch.zeros_like(buf, dtype=torch.bool)
    torch.as_strided(inside, view.shape, view.stride(), view.storage_offset()).fill_(True)
    return bool((~inside).any()) and bool(torch.isnan(buf[~inside]).all())


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("shift,pad", [(0, 8), (8, 16), (4, 4), (1, 3)])
@pytest.mark.parametrize("rows,d,f,experts", [(5, 72, 200, 0), (12, 72, 200, 0), (140, 72, 200, 0), (140, 50, 24, 0), (3000, 1000, 520, 0),
                                              (300, 104, 72, 64), (3400, 264, 280, 48), (4200, 264, 280, 0)])
def test_nothing_beside_the_results(spmv, dtype, shift, pad, rows, d, f, experts):
    """every array that the block writes, gate and up, both workspaces and the weights' gradients among them, with NaN between its
    rows and around it: what was there stays, and the results are those of the plain call"""
    g = gen(rows + pad)
    lead = experts or None
    if experts:
        plan, x, dy, _ = routed(spmv, rows, 1, experts, 1, d, dtype, g)
        x, dy = placed(x.cpu(), shift, pad), placed(dy.cpu(), shift, pad)
        want = plan.feed_forward(x, *(ws := weights(lead, d, f, dtype, g, shift, pad)), keep=True)
    else:
        x, dy = (placed(torch.randn(rows, d, generator=g).to(dtype), shift, pad) for _ in range(2))
        want = spmv.feed_forward(x, *(ws := weights(lead, d, f, dtype, g, shift, pad)), keep=True)
    rows = len(x)
    want_grad = want.grad(dy)
    code = {torch.float32: 1, torch.float16: 2, torch.bfloat16: 3}[dtype]
    (y, y_all), (dx, dx_all) = (guarded((rows, d), dtype, shift, pad) for _ in range(2))
    (gate, gate_all), (up, up_all) = (guarded((rows, f), dtype, shift, pad) for _ in range(2))
    dws = [guarded(w.shape, dtype, 8) for w in ws]  # (contiguous, in front of a row's worth of values)
    spaces = []
    for gradient in (0, 1):
        n = spmv.spmv_feed_forward_workspace(rows, d, f, experts or 1, code, gradient)
        spaces.append((n, torch.full((n + 512,), 0x5a, dtype=torch.uint8, device="cuda")))
    apart = [w.stride(0) if experts else 0 for w in ws]
    call = (rows, d, f, experts or 1, plan.offsets if experts else None, x, x.stride(0), ws[0], ws[1], ws[0].stride(-2), apart[0], ws[2],
            ws[2].stride(-2), apart[2], "silu", gate, up, gate.stride(0))
    spmv.spmv_feed_forward(*call, y, y.stride(0), code, spaces[0][1][256:], spaces[0][0])
    spmv.spmv_feed_forward_grad(*call, dy, dy.stride(0), dx, dx.stride(0), *[v for v, _ in dws], code, spaces[1][1][256:], spaces[1][0])
    for name, view, buf in (("y", y, y_all), ("dx", dx, dx_all), ("gate", gate, gate_all), ("up", up, up_all),
                            *((f"dw{i}", *pair) for i, pair in enumerate(dws))):
        assert untouched(view, buf), name
    for n, space in spaces:
        assert space[:256].eq(0x5a).all() and space[256 + n:].eq(0x5a).all()
    for name, got, ref_ in (("gate", gate, want.gate), ("up", up, want.up), ("y", y, want.y), ("dx", dx, want_grad[0]),
                            *((f"dw{i}", v, w) for i, ((v, _), w) in enumerate(zip(dws, want_grad[1:])))):
        assert torch.equal(got, ref_), name


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("rows", [2, 20])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_large_gates_of_other_types(spmv, dtype, rows, act):
    """gates up to the end of the type's range, or of the exponential's: act tends to x or to 0, no NaN"""
    scale = [0.0, 1.0, 20.0, 90.0, 1e4, 6e4, -20.0, -90.0] if dtype == torch.float16 else [0.0, 1.0, 20.0, 90.0, 1e4, 1e15, 1e18, -1e18]
    x = torch.tensor([1.0, -1.0]).repeat(rows // 2)[:, None].repeat(1, 8).to(dtype).cuda()
    wg, wu = torch.zeros(8, 8, dtype=dtype), torch.zeros(8, 8, dtype=dtype)
    wg[:, 0], wu[:, 0] = torch.tensor(scale).to(dtype), 1.0
    ws = (wg.cuda(), wu.cuda(), torch.eye(8, dtype=dtype, device="cuda"))
    dy = torch.ones_like(x)
    res = spmv.feed_forward(x, *ws, activation=act, keep=True)
    dx, dwg, dwu, dwd = res.grad(dy)
    kw = dict(unit=U, half=H[dtype], tiny=TINY[dtype])
    w = [f64(t) for t in ws]
    fwd = ref.feed_forward(f64(x), *w, act, **kw)
    back = ref.feed_forward_grad(f64(x), *w, act, f64(res.gate), f64(res.up), f64(dy), **kw)
    for got, (want, bound) in ((res.gate, fwd["gate"]), (res.up, fwd["up"]), (res.y, fwd["y"]), (dx, back["dx"]), (dwg, back["dw_gate"]),
                               (dwu, back["dw_up"]), (dwd, back["dw_down"])):
        beyond = np.abs(want) - bound > torch.finfo(dtype).max  # (a sum of gradients beyond the type's range is an infinity)
        got = f64(got)
        assert np.array_equal(got[beyond], np.copysign(np.inf, want[beyond]))
        assert (np.abs(got - want) <= bound)[~beyond].all()


@pytest.mark.parametrize("rows", [4, 12, 40])
def test_values_beyond_float16(spmv, rows):
    """h is a value of the type: beyond 65504 it is an infinity, in y an infinity or (beside a 0 of w_down) NaN, in its row only"""
    x = torch.ones(rows, 16, dtype=torch.float16, device="cuda")
    x[::2] = 0.125
    wg, wu, wd = (torch.zeros(16, 16, dtype=torch.float16, device="cuda") for _ in range(3))
    wg[0, 0] = wu[0, 0] = 300.0
    wd[3, 0] = 0.5
    y = spmv.feed_forward(x, wg, wu, wd).y
    assert torch.isinf(y[1::2, 3]).all() and torch.isnan(y[1::2, 4]).all()
    assert torch.equal(y[::2, 3], torch.full_like(y[::2, 3], 37.5 * 37.5 / 2)) and not y[::2, 4].any()
