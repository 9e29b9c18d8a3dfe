"""What the table lookup and the feed-forward block refuse, and what their Python functions hand on: nothing
runs on a GPU (host arrays stand in for device ones, or the library is stood in for)."""
import numpy as np
import pytest
import torch

F32, F16, BF16 = 1, 2, 3


@pytest.fixture(scope="module")
def spmv():
    import __graft_entry__

    __graft_entry__._build_module().build()
    import sparse_matrix_vector_csr_gb300 as spmv

    return spmv


def status(spmv, call, *args, **kw):
    with pytest.raises(spmv.SpmvError) as e:
        call(*args, **kw)
    return e.value.status, str(e.value)


def test_lookup_refusals(spmv):
    h = np.zeros(64, np.float32)
    ok = dict(tokens=2, vocab=4, d=3, ids=h, table=h, ldtable=3, scale=1.0, x=h, ldx=3, dtype=F32, stream=0)
    for change, word in (({"tokens": -1}, "tokens"), ({"tokens": 1 << 31}, "tokens"), ({"vocab": 0}, "vocab"), ({"d": -1}, "d must"),
                         ({"dtype": 0}, "dtype"), ({"ids": None}, "ids"), ({"ids": h.ctypes.data + 2}, "ids"), ({}, "ids is not device")):
        s, text = status(spmv, spmv.spmv_embed_rows, **{**ok, **change})
        assert s == -1 and word in text, (change, text)
    assert status(spmv, spmv.spmv_embed_rows, **{**ok, "tokens": (1 << 31) - 1, "d": 1 << 20})[0] == -5
    spmv.spmv_embed_rows(**{**ok, "tokens": 0, "ids": None, "table": None, "x": None})
    assert status(spmv, spmv.spmv_embed_workspace, 5, 0, 4)[0] == -1
    assert spmv.spmv_embed_workspace(0, 4, 8) >= 4
    one, two = spmv.spmv_embed_workspace(1000, 512, 64), spmv.spmv_embed_workspace(1000, 513, 64)
    assert two - one == 8000  # a second pass keeps keys and places of its own


def test_gradient_refusals(spmv):
    h = np.zeros(64, np.float32)
    ok = dict(tokens=2, vocab=4, d=3, ids=h, dx=h, lddx=3, dtype=F16, scale=1.0, accumulate=0, dtable=h, lddtable=3,
              out_dtype=F16, workspace=h, workspace_bytes=256, stream=0)
    for change, word in (({"out_dtype": BF16}, "out_dtype"), ({"out_dtype": 0}, "out_dtype"), ({"workspace_bytes": 8}, "workspace"),
                         ({"lddtable": 2}, "leading"), ({"dtable": None}, "dtable"), ({}, "not device")):
        s, text = status(spmv, spmv.spmv_embed_rows_grad, **{**ok, **change})
        assert s == -1 and word in text, (change, text)
    spmv.spmv_embed_rows_grad(**{**ok, "tokens": 0, "accumulate": 1, "dtable": None})  # nothing to add


FF = dict(rows=2, d=8, f=8, experts=1, offsets=None, ldx=8, ldw=8, w_expert=64, ldwd=8, wd_expert=64, activation="silu", ldg=8,
          dtype=BF16, workspace_bytes=1 << 12, stream=0)


def test_feed_forward_refusals(spmv):
    h = np.zeros(256, np.float32)
    arrays = dict(x=h, w_gate=h, w_up=h, w_down=h, gate=None, up=None, y=h, ldy=8, workspace=h)
    for change, word in (({"rows": -1}, "rows"), ({"d": 0}, "d and f"), ({"f": (1 << 20) + 1}, "d and f"), ({"dtype": 0}, "dtype"),
                         ({"activation": 7}, "activation"), ({"gate": h}, "gate and up"), ({"experts": 0}, "experts"),
                         ({"experts": 4097, "offsets": h}, "experts"), ({"experts": 2}, "offsets"), ({"workspace_bytes": 8}, "workspace"),
                         ({"ldx": 7}, "x: the leading"), ({}, "x is not device")):
        s, text = status(spmv, spmv.spmv_feed_forward, **{**FF, **arrays, **change})
        assert s == -1 and word in text, (change, text)
    spmv.spmv_feed_forward(**{**FF, **arrays, "rows": 0, "x": None, "y": None})
    assert spmv.spmv_feed_forward_workspace(3, 8, 9, 1, BF16) == 2 * 3 * 16 * 2  # (few rows: h in two parts)
    assert spmv.spmv_feed_forward_workspace(17, 8, 9, 1, BF16) == 17 * 16 * 2 == spmv.spmv_feed_forward_workspace(17, 8, 9, 2, BF16)
    assert spmv.spmv_feed_forward_workspace(3, 8, 9, 1, F32, True) == 3 * 3 * 16 * 4
    back = dict(x=h, w_gate=h, w_up=h, w_down=h, gate=h, up=h, dy=h, lddy=8, dx=h, lddx=8, dw_gate=h, dw_up=h, dw_down=h, workspace=h)
    for change, word in (({"experts": 2}, "offsets"), ({"activation": -1}, "activation"), ({}, "x is not device")):
        s, text = status(spmv, spmv.spmv_feed_forward_grad, **{**FF, **back, **change})
        assert s == -1 and word in text, (change, text)


@pytest.fixture
def rows(spmv, monkeypatch):
    """The Python functions over a library that notes its calls and succeeds."""
    from sparse_matrix_vector_csr_gb300 import sparse_rows

    class Recorder:
        def __init__(self, lib):
            self.lib, self.calls = lib, []

        def __getattr__(self, name):
            if name.endswith(("_workspace", "_route_rows")):
                return getattr(self.lib, name)
            return lambda *args: self.calls.append((name, args)) or 0

    monkeypatch.setattr(sparse_rows, "lib", Recorder(sparse_rows.lib))
    return sparse_rows


def test_embed_rows_arguments(rows):
    table, ids = torch.zeros(6, 8, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    dx = torch.zeros(3, 8, dtype=torch.float16)
    assert rows.embed_rows(table, ids).shape == (3, 8)
    assert rows.embed_rows_grad(dx, ids, 6).dtype == torch.float16
    assert rows.embed_rows_grad(dx, ids, 6, dtype=torch.float32).dtype == torch.float32
    for bad, error in ((lambda: rows.embed_rows(table.double(), ids), TypeError), (lambda: rows.embed_rows(table, ids.long()), TypeError),
                       (lambda: rows.embed_rows(table, ids[:, None]), ValueError), (lambda: rows.embed_rows(table.t(), ids), ValueError),
                       (lambda: rows.embed_rows(table, ids, out=torch.zeros(3, 7, dtype=torch.float16)), ValueError),
                       (lambda: rows.embed_rows_grad(dx, ids[:2], 6), ValueError),
                       (lambda: rows.embed_rows_grad(dx, ids, 6, accumulate=True), ValueError),
                       (lambda: rows.embed_rows_grad(dx, ids, 6, dtype=torch.bfloat16), TypeError),
                       (lambda: rows.embed_rows_grad(dx, ids, 6, out=table.float(), dtype=torch.float16), TypeError),
                       (lambda: rows.embed_rows_grad(dx, ids, 5, out=table), ValueError)):
        with pytest.raises(error):
            bad()


def test_feed_forward_arguments(rows):
    x, wg, wu, wd = torch.zeros(5, 8), torch.zeros(12, 8), torch.zeros(12, 8), torch.zeros(8, 12)
    assert rows.feed_forward(x, wg, wu, wd).y.shape == (5, 8)
    with pytest.raises(ValueError, match="keep"):
        rows.feed_forward(x, wg, wu, wd).grad(x)
    res = rows.feed_forward(x, wg, wu, wd, keep=True)
    assert res.gate.shape == (5, 12) and res.gate.stride(0) == 16  # 16-byte rows whatever f is
    assert [t.shape for t in res.grad(x)] == [x.shape, wg.shape, wu.shape, wd.shape]
    assert res.grad(x, weights=False)[1:] == (None, None, None)
    fused = torch.zeros(24, 8)
    rows.feed_forward(x, fused[:12], fused[12:], wd)
    for bad, error in ((lambda: rows.feed_forward(x, wg.half(), wu, wd), TypeError), (lambda: rows.feed_forward(x, wg, wu[:11], wd), ValueError),
                       (lambda: rows.feed_forward(x, wg, torch.zeros(12, 9)[:, :8], wd), ValueError),
                       (lambda: rows.feed_forward(x, wg, wu, wd.t()), ValueError), (lambda: rows.feed_forward(x, wg[None], wu[None], wd[None]), ValueError),
                       (lambda: rows.feed_forward(x, wg, wu, wd, activation="tanh"), KeyError)):
        with pytest.raises(error):
            bad()


def test_experts_feed_forward_arguments(rows):
    plan = rows.RoutePlan(torch.zeros(6, 2, dtype=torch.int32), 4, align=2)
    xs, fused, wd = torch.zeros(plan.rows, 8), torch.zeros(4, 24, 8), torch.zeros(4, 8, 12)
    rows.lib.calls.clear()
    plan.feed_forward(xs, fused[:, :12], fused[:, 12:], wd)
    (name, args), = rows.lib.calls
    assert name == "spmv_feed_forward" and args[:5] == (plan.rows, 8, 12, 4, plan.offsets.data_ptr())
    assert args[9:11] == (8, 24 * 8) and args[12:14] == (12, 96)
    for bad in (lambda: plan.feed_forward(xs[:-1], fused[:, :12], fused[:, 12:], wd), lambda: plan.feed_forward(xs, fused[:3, :12], fused[:3, 12:], wd),
                lambda: plan.feed_forward(xs, fused[0, :12], fused[0, 12:], wd[0]),
                lambda: plan.feed_forward(xs, fused[:, :12].expand(4, 12, 8), fused[:, 12:], wd[:1].expand(4, 8, 12))):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("change", ["none", "deepcopy", "pickle", "assigned"])
def test_a_block_passes_the_tensors_it_has(rows, change):
    """the gradient's call gets the addresses of the tensors that the result holds, copied or not; other tensors
    in the public attributes change nothing"""
    import copy
    import pickle

    plan = rows.RoutePlan(torch.zeros(6, 2, dtype=torch.int32), 4, align=2)
    xs, w, wd = torch.zeros(plan.rows, 8), [torch.zeros(4, 12, 8) for _ in range(2)], torch.zeros(4, 8, 12)
    res = kept = plan.feed_forward(xs, *w, wd, keep=True)
    if change == "deepcopy":
        res = copy.deepcopy(res)
    elif change == "pickle":
        res = pickle.loads(pickle.dumps(res))
    elif change == "assigned":
        res.gate, plan.offsets = torch.ones_like(res.gate), torch.ones_like(plan.offsets)
    rows.lib.calls.clear()
    res.grad(xs)
    (name, args), = rows.lib.calls
    x, wg, wu, wdown, offsets, _, gate, up, _ = res._args
    assert name == "spmv_feed_forward_grad"
    assert [args[i] for i in (4, 5, 7, 8, 11, 15, 16)] == [t.data_ptr() for t in (offsets, x, wg, wu, wdown, gate, up)]
    assert (x.data_ptr() == xs.data_ptr()) == (change in ("none", "assigned")) and args[15] != (res.gate if change == "assigned" else x).data_ptr()
    del kept
