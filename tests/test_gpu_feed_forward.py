"""The gated feed-forward block over segments on the GPU against its 64-bit statement (oracle/token_rows.py).

Tolerances are elementwise and come from the arithmetic: a sum of n products in 32 bits is within n U of the
terms' magnitudes (U = 2^-23: products are exact, additions may be cut off instead of rounded), a rounding to the
type within H of the value (half a step) or half the smallest step, and what h's and the gradients' roundings do
to the next product is carried through with absolute values.
"""
import math

import numpy as np
import pytest
import torch

from oracle import token_rows as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
H = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -25, torch.bfloat16: 1e-37}
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


def placed(t, shift=0, pad=0):
    """t at an address `shift` values behind an aligned one, its rows `pad` values apart, NaN around them."""
    lead, n = t.shape[:-1], t.shape[-1]
    rows = math.prod(lead)
    buf = torch.full((shift + rows * (n + pad) + 8,), math.nan, dtype=t.dtype, device="cuda")
    view = buf[shift:shift + rows * (n + pad)].view(*lead, n + pad)[..., :n]
    view.copy_(t)
    return view


def weights(experts, d, f, dtype, g, shift=0, pad=0):
    lead = () if experts is None else (experts,)
    wg = (torch.randn(*lead, f, d, generator=g) * d ** -0.5).to(dtype)
    wu = (torch.randn(*lead, f, d, generator=g) * d ** -0.5).to(dtype)
    wd = (torch.randn(*lead, d, f, generator=g) * f ** -0.5).to(dtype)
    return [placed(w, shift, pad) for w in (wg, wu, wd)]


def within(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3], bound[bad][:3])


def check(spmv, x, ws, act, dy, spans, run):
    """forward and back of blocks over the spans [(begin, end)] of x, one a matrix of ws"""
    dtype = x.dtype
    kw = dict(unit=U, half=H[dtype], tiny=TINY[dtype])
    res = run(keep=True)
    dx, dwg, dwu, dwd = res.grad(dy)
    plain = run(keep=False)
    assert torch.equal(plain.y, res.y)
    end = 0
    for e, (a, end) in enumerate(spans):
        w = [f64(t[e] if t.dim() == 3 else t) for t in ws]
        xe = f64(x[a:end])
        fwd = ref.feed_forward(xe, *w, act, **kw)
        for name, got in (("gate", res.gate), ("up", res.up), ("y", res.y)):
            within(got[a:end], *fwd[name], (name, e))
        back = ref.feed_forward_grad(xe, *w, act, f64(res.gate[a:end]), f64(res.up[a:end]), f64(dy[a:end]), **kw)
        within(dx[a:end], *back["dx"], ("dx", e))
        for name, got in (("dw_gate", dwg), ("dw_up", dwu), ("dw_down", dwd)):
            within(got[e] if got.dim() == 3 else got, *back[name], (name, e))
    for name, got in (("y", res.y), ("gate", res.gate), ("up", res.up), ("dx", dx)):
        assert not got[end:].any(), name
    again = res.grad(dy)
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dwg, dwu, dwd)))  # the same bits every time
    only = res.grad(dy, weights=False)
    assert torch.equal(only[0], dx) and only[1:] == (None, None, None)
    return res, (dx, dwg, dwu, dwd)


SIZES = [(1, 1, 1), (3, 5, 7), (1, 8, 8), (5, 64, 40), (128, 128, 128), (129, 136, 72), (257, 520, 264), (64, 37, 53),
         (300, 1000, 96), (40, 24, 1032), (1000, 64, 64), (33, 512, 768)]


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,d,f", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_dense(spmv, dtype, rows, d, f, act):
    g = gen(rows + d + f)
    x, dy = torch.randn(rows, d, generator=g).to(dtype).cuda(), torch.randn(rows, d, generator=g).to(dtype).cuda()
    ws = weights(None, d, f, dtype, g)
    check(spmv, x, ws, act, dy, [(0, rows)], lambda keep: spmv.feed_forward(x, *ws, activation=act, keep=keep))


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 0), (3, 5), (8, 16), (4, 4), (2, 6)])
@pytest.mark.parametrize("d,f", [(72, 200), (50, 24)])
def test_any_address(spmv, dtype, shift, pad, d, f):
    g = gen(d + pad)
    x, dy = (placed(torch.randn(140, d, generator=g).to(dtype), shift, pad) for _ in range(2))
    ws = weights(None, d, f, dtype, g, shift, pad)
    y, dx = (placed(torch.zeros(140, d, dtype=dtype), pad, shift) for _ in range(2))
    res, grads = check(spmv, x, ws, "silu", dy, [(0, 140)], lambda keep: spmv.feed_forward(x, *ws, keep=keep))
    into = spmv.feed_forward(x, *ws, keep=True, out=y)
    assert into.y is y and torch.equal(y, res.y)
    assert into.grad(dy, out=dx)[0] is dx and torch.equal(dx, grads[0])
    for t in (y, dx):  # nothing beside the rows
        whole = torch.as_strided(t, (140 * t.stride(0) + 8,), (1,), 0) if t.storage_offset() == 0 else None
        if whole is not None:
            outside = torch.ones_like(whole, dtype=torch.bool)
            torch.as_strided(outside, t.shape, t.stride(), 0).fill_(False)
            assert bool(torch.isnan(whole[outside]).all())


def routed(spmv, tokens, k, experts, align, d, dtype, g, only=None, dropped=0.1):
    ids = torch.rand(tokens, experts, generator=g).topk(k, dim=1).indices.to(torch.int32)
    if only is not None:
        ids = only[ids.long() % len(only)]
    ids = torch.where(torch.rand(tokens, k, generator=g) < dropped, torch.full_like(ids, -1), ids).cuda()
    plan = spmv.RoutePlan(ids, experts, align=align)
    xs = plan.dispatch(torch.randn(tokens, d, generator=g).to(dtype).cuda())
    dys = plan.dispatch(torch.randn(tokens, d, generator=g).to(dtype).cuda())
    offsets = plan.offsets.tolist()
    end = offsets[-1]
    xs[end:], dys[end:] = math.nan, math.nan  # rows without an expert: not looked at
    return plan, xs, dys, list(zip(offsets, offsets[1:]))


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("tokens,k,experts,align,d,f", [(1, 1, 1, 1, 16, 8), (1, 2, 4, 1, 64, 64), (7, 3, 9, 1, 48, 40),
                                                        (60, 2, 5, 16, 72, 136), (400, 2, 3, 128, 128, 256),
                                                        (333, 3, 17, 1, 136, 104), (90, 4, 64, 4, 64, 32), (50, 2, 7, 1, 45, 31),
                                                        (900, 1, 2, 1, 264, 72)])
def test_experts(spmv, dtype, tokens, k, experts, align, d, f):
    g = gen(tokens + experts)
    plan, xs, dys, spans = routed(spmv, tokens, k, experts, align, d, dtype, g)
    ws = weights(experts, d, f, dtype, g)
    check(spmv, xs, ws, "silu", dys, spans, lambda keep: plan.feed_forward(xs, *ws, keep=keep))


@pytest.mark.parametrize("dtype", ALL)
def test_experts_without_rows_and_all_in_one(spmv, dtype):
    g = gen(3)
    for only in (torch.tensor([5], dtype=torch.int32), torch.tensor([0, 7], dtype=torch.int32), torch.tensor([-1], dtype=torch.int32)):
        plan, xs, dys, spans = routed(spmv, 150, 2, 8, 1, 64, dtype, g, only)
        ws = weights(8, 64, 72, dtype, g)
        _, grads = check(spmv, xs, ws, "gelu_tanh", dys, spans,
                         lambda keep: plan.feed_forward(xs, *ws, activation="gelu_tanh", keep=keep))
        for e, (a, b) in enumerate(spans):
            if a == b:
                assert not any(t[e].any() for t in grads[1:])


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,d,f", [(1024, 64, 64), (2500, 40, 136), (5000, 37, 53), (4133, 8, 8), (1100, 264, 72)])
def test_many_rows_of_small_matrices(spmv, dtype, rows, d, f):
    """the weights' gradients in several parts of the rows"""
    g = gen(rows)
    x, dy = torch.randn(rows, d, generator=g).to(dtype).cuda(), torch.randn(rows, d, generator=g).to(dtype).cuda()
    ws = weights(None, d, f, dtype, g)
    check(spmv, x, ws, "silu", dy, [(0, rows)], lambda keep: spmv.feed_forward(x, *ws, keep=keep))


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("align,d,f", [(1, 64, 40), (16, 72, 128), (1, 21, 30)])
def test_experts_of_many_rows(spmv, dtype, align, d, f):
    """parts of segments of different lengths, one of them empty, one of a few rows"""
    g = gen(align + d)
    ids = torch.tensor([0] * 3000 + [2] * 1500 + [3] * 7, dtype=torch.int32)[torch.randperm(4507, generator=g)][:, None].cuda()
    plan = spmv.RoutePlan(ids, 4, align=align)
    xs, dys = (plan.dispatch(torch.randn(4507, d, generator=g).to(dtype).cuda()) for _ in range(2))
    offsets = plan.offsets.tolist()
    xs[offsets[-1]:], dys[offsets[-1]:] = math.nan, math.nan
    ws = weights(4, d, f, dtype, g)
    _, grads = check(spmv, xs, ws, "silu", dys, list(zip(offsets, offsets[1:])), lambda keep: plan.feed_forward(xs, *ws, keep=keep))
    assert not any(w[1].any() for w in grads[1:])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_wide_tiles(spmv, dtype):
    """sizes at which pairs of CTAs share a tile, in the forward and every backward product, ragged at every border; against
    products in 64 bits on the GPU"""
    g = gen(11)
    plan, xs, dys, spans = routed(spmv, 1500, 2, 3, 1, 1032, dtype, g)
    ws = weights(3, 1032, 4104, dtype, g)
    ff = plan.feed_forward(xs, *ws, keep=True)
    grads = ff.grad(dys)
    for e, (a, b) in enumerate(spans):
        leaves = [t.double().requires_grad_() for t in (xs[a:b], *(w[e] for w in ws))]
        gate, up = leaves[0] @ leaves[1].t(), leaves[0] @ leaves[2].t()
        y = (torch.nn.functional.silu(gate) * up) @ leaves[3].t()
        want = [gate, up, y, *torch.autograd.grad(y, leaves, dys[a:b].double())]
        got = [ff.gate[a:b], ff.up[a:b], ff.y[a:b], grads[0][a:b], *(w[e] for w in grads[1:])]
        for i, (p, q) in enumerate(zip(got, want)):
            # roundings, each within H of a value: of the result; of h (y); of gate, up and their gradients (the others)
            assert float((p.double() - q).norm() / q.norm()) <= H[dtype] * (1, 1, 2, 4, 4, 4, 4)[i], i
            assert float((p.double() - q).abs().max()) <= H[dtype] * 8 * float(q.abs().max()), i


@pytest.mark.parametrize("dtype,d,f", [(torch.bfloat16, 64, 72), (torch.float32, 30, 21)])
def test_offsets_of_no_plan(spmv, dtype, d, f):
    """offsets that no plan gives (out of range, falling): spans are cut to the rows, nothing beside the rows is
    written.  (Rows in two spans have no one result.)"""
    g = gen(12)
    rows, experts = 150, 4
    xs, dys = (torch.randn(rows, d, generator=g).to(dtype).cuda() for _ in range(2))
    ws = weights(experts, d, f, dtype, g)
    plan = spmv.RoutePlan(torch.zeros(rows, 1, dtype=torch.int32, device="cuda"), experts)
    for values in ([0, 40, 30, 2 ** 31 - 1, -5], [-3, -2, -1, 0, 10 ** 9], [149, 149, 149, 149, 149], [2 ** 31 - 1] * 5):
        plan.offsets = torch.tensor(values, dtype=torch.int32).cuda()
        around = [torch.full((rows + 20, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        res = plan.feed_forward(xs, *ws, keep=True, out=around[0][10:-10])
        res.grad(dys, out=around[1][10:-10])
        for t in around:
            assert t[:10].eq(7).all() and t[-10:].eq(7).all() and torch.isfinite(t).all()
    assert res.y.eq(7).all()  # (the last: every row lies in front of the first segment, and is left as it was)
    spmv.spmv_feed_forward_status()


def test_status(spmv):
    """no wait of any call before has run out"""
    spmv.spmv_feed_forward_status()


def test_many_experts(spmv):
    g = gen(4)
    ids = torch.randint(0, 4096, (300, 2), generator=g, dtype=torch.int32).cuda()
    plan = spmv.RoutePlan(ids, 4096)
    xs = plan.dispatch(torch.randn(300, 16, generator=g).bfloat16().cuda())
    ws = weights(4096, 16, 8, torch.bfloat16, g)
    y = plan.feed_forward(xs, *ws).y
    e = torch.repeat_interleave(torch.arange(4096), plan.offsets.cpu().diff())
    for r in range(0, 600, 37):
        out = ref.feed_forward(f64(xs[r:r + 1]), *[f64(w[e[r]]) for w in ws], "silu", unit=U, half=H[torch.bfloat16], tiny=1e-37)
        within(y[r:r + 1], *out["y"], r)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("d,f", [(64, 136), (45, 50)])
def test_bad_values_stay_in_their_row(spmv, dtype, d, f):
    """NaN and infinities of a row reach its own results and its expert's weight gradients, nothing else"""
    g = gen(5)
    plan, xs, dys, spans = routed(spmv, 200, 2, 4, 1, d, dtype, g, dropped=0.0)
    ws = weights(4, d, f, dtype, g)
    clean = plan.feed_forward(xs, *ws, keep=True)
    want = clean.grad(dys)
    bad = xs.clone()
    row = spans[1][0] + 2
    bad[row, 3], bad[row, 5] = math.nan, math.inf
    got = plan.feed_forward(bad, *ws, keep=True)
    back = got.grad(dys)
    rest = torch.arange(len(xs), device="cuda") != row
    assert torch.isnan(got.y[row]).all()
    assert torch.equal(got.y[rest], clean.y[rest]) and torch.equal(back[0][rest], want[0][rest])
    for p, q in zip(back[1:], want[1:]):
        assert all(torch.equal(p[e], q[e]) for e in (0, 2, 3)) and torch.isnan(p[1]).any()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_large_gates(spmv, act):
    """gates at both ends of the exponential's range: act tends to x or to 0, no NaN"""
    x = torch.tensor([[1.0], [-1.0]]).repeat(1, 8).bfloat16().cuda()
    scale = torch.tensor([0.0, 1.0, 20.0, 90.0, 1e4, 1e15, 1e18, -1e18]).bfloat16()
    wg = torch.zeros(8, 8, dtype=torch.bfloat16)
    wg[:, 0] = scale
    wu, wd = torch.zeros(8, 8, dtype=torch.bfloat16), torch.eye(8, dtype=torch.bfloat16)
    wu[:, 0] = 1.0
    wg, wu, wd = wg.cuda(), wu.cuda(), wd.cuda()
    dy = torch.ones(2, 8, dtype=torch.bfloat16, device="cuda")
    check(spmv, x, (wg, wu, wd), act, dy, [(0, 2)], lambda keep: spmv.feed_forward(x, wg, wu, wd, activation=act, keep=keep))


def test_fused_weights_and_no_rows(spmv):
    g = gen(6)
    fused = (torch.randn(3, 2 * 72, 64, generator=g) / 8).bfloat16().cuda()
    wd = (torch.randn(3, 64, 72, generator=g) / 8).bfloat16().cuda()
    plan, xs, dys, spans = routed(spmv, 80, 2, 3, 1, 64, torch.bfloat16, g)
    ws = (fused[:, :72], fused[:, 72:], wd)
    check(spmv, xs, ws, "silu", dys, spans, lambda keep: plan.feed_forward(xs, *ws, keep=keep))
    none = spmv.feed_forward(xs[:0], *[w[0] for w in ws], keep=True)
    assert none.y.shape == (0, 64)
    dx, *dws = none.grad(xs[:0])
    assert dx.shape == (0, 64) and not any(w.any() for w in dws)


def test_gradient_against_differences(spmv):
    """Central differences of <dy, y> in float, along random directions of every input."""
    g = gen(7)
    x, dy = torch.randn(20, 24, generator=g).cuda(), torch.randn(20, 24, generator=g).cuda()
    ws = [w.contiguous() for w in weights(None, 24, 40, torch.float32, g)]
    for act in ("silu", "gelu_tanh"):
        grads = spmv.feed_forward(x, *ws, activation=act, keep=True).grad(dy)
        for i in range(4):
            args = [x, *ws]
            v, step = torch.randn(args[i].shape, generator=g).cuda(), 2.0 ** -6

            def value(h):
                moved = list(args)
                moved[i] = args[i] + h * v
                return float((spmv.feed_forward(*moved, activation=act).y.double() * dy.double()).sum())

            # fourth-order differences: error of step^4 times the fifth derivative, and rounding / step
            slope = (8 * (value(step) - value(-step)) - (value(2 * step) - value(-2 * step))) / (12 * step)
            assert abs(slope - float((grads[i].double() * v.double()).sum())) <= 2e-3 * float((grads[i] * v).abs().sum() / len(v) ** 0.5 + 1), (act, i)


def test_streams_and_graph(spmv):
    g = gen(8)
    plan, xs, dys, _ = routed(spmv, 500, 2, 6, 1, 128, torch.bfloat16, g, dropped=0.0)
    ws = weights(6, 128, 192, torch.bfloat16, g)
    want = plan.feed_forward(xs, *ws, keep=True)
    want_grad = want.grad(dys)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = plan.feed_forward(xs, *ws, keep=True, stream=side)
    got_grad = got.grad(dys, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got.y, want.y) and all(torch.equal(p, q) for p, q in zip(got_grad, want_grad))
    x, dy = torch.zeros_like(xs), torch.zeros_like(dys)
    graphs = []
    for _ in range(2):  # two graphs of the same call, each with its own workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = plan.feed_forward(x, *ws, keep=True)
            grads = res.grad(dy)
        graphs.append((graph, res, grads))
    for scale in (1.0, -0.5):
        x.copy_(xs * scale), dy.copy_(dys)
        for graph, _, _ in graphs:
            graph.replay()
        now = plan.feed_forward(x, *ws, keep=True)
        now_grad = now.grad(dy)
        for _, res, grads in graphs:
            assert torch.equal(res.y, now.y) and all(torch.equal(p, q) for p, q in zip(grads, now_grad))


def test_two_calls_at_once(spmv):
    """blocks of different sizes on two streams, over and over, each with the results of its own run"""
    g = gen(9)
    sets = []
    for rows, d, f in ((700, 256, 512), (90, 512, 128)):
        x = torch.randn(rows, d, generator=g).bfloat16().cuda()
        ws = weights(None, d, f, torch.bfloat16, g)
        sets.append((x, ws, spmv.feed_forward(x, *ws).y, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [(want, spmv.feed_forward(x, *ws, stream=s).y) for _ in range(20) for x, ws, want, s in sets]
    torch.cuda.synchronize()
    assert all(torch.equal(want, got) for want, got in outs)


def test_a_layer_from_tokens_to_tokens(spmv):
    """Lookup, router, experts and back, forward and gradients, against the same layer under autograd in 64
    bits (float throughout: the two differ by rounding)."""
    g = gen(10)
    n, vocab, d, f, experts, k = 70, 40, 48, 56, 5, 2
    table, router = torch.randn(vocab, d, generator=g).cuda(), (torch.randn(d, experts, generator=g) / 7).cuda()
    ws = [w.contiguous() for w in weights(experts, d, f, torch.float32, g)]
    ids = torch.randint(0, vocab, (n,), generator=g, dtype=torch.int32).cuda()
    dy = torch.randn(n, d, generator=g).cuda()

    x = spmv.embed_rows(table, ids, scale=2.0)
    top = spmv.topk_rows(x @ router, k, weights="selected")
    plan = spmv.RoutePlan(top.ids, experts, align=8)
    ff = plan.feed_forward(plan.dispatch(x), *ws, keep=True)
    y = plan.combine(ff.y, top.weights)
    dys, dweights = plan.combine_grad(dy, ff.y, top.weights)
    dxs, *dws = ff.grad(dys)
    dx = plan.dispatch_grad(dxs) + top.grad(dweights) @ router.t()
    got = [spmv.embed_rows_grad(dx, ids, vocab, scale=2.0), *dws]

    leaves = [t.double().requires_grad_() for t in (table, *ws)]
    e = leaves[0][ids.long()] * 2.0
    val, at = (e @ router.double()).topk(k, dim=1)
    assert torch.equal(at.to(torch.int32), top.ids)
    p = torch.softmax(val, 1)
    out = 0
    for j in range(k):
        wg, wu, wd = (w[at[:, j]] for w in leaves[1:])
        h = torch.nn.functional.silu(torch.einsum("td,tfd->tf", e, wg)) * torch.einsum("td,tfd->tf", e, wu)
        out = out + p[:, j:j + 1] * torch.einsum("tf,tdf->td", h, wd)
    assert (y.double() - out).abs().max() <= 1e-4 * out.abs().max()
    want = torch.autograd.grad(out, leaves, dy.double())
    for p, q in zip(got, want):
        assert (p.double() - q).abs().max() <= 1e-4 * q.abs().max()
