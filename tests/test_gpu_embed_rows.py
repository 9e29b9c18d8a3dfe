"""Rows of a table by token and their gradient on the GPU against 64-bit statements (oracle/token_rows.py).

A lookup is exact, or one rounding of a product (half a step: H).  A gradient's sum of n terms in 32 bits is
within n E of the terms' magnitudes (E = 2^-24), the product with the scale adds E, the type's rounding H.
"""
import math

import numpy as np
import pytest
import torch

from oracle import token_rows as ref

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
H = {torch.float32: E, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -25, torch.bfloat16: 1e-37}
ALL = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def spmv():
    import __graft_entry__

    __graft_entry__._build_module().build()
    import sparse_matrix_vector_csr_gb300 as spmv

    return spmv


def placed(t, shift=0, pad=0):
    """t at an address `shift` values behind an aligned one, rows `pad` values apart, NaN around them."""
    rows, n = t.shape
    buf = torch.full((shift + rows * (n + pad) + 8,), math.nan, dtype=t.dtype, device="cuda")
    view = buf[shift:shift + rows * (n + pad)].view(rows, n + pad)[:, :n]
    view.copy_(t)
    return view, buf


def untouched(view, buf):
    inside = torch.zeros_like(buf, dtype=torch.bool)
    torch.as_strided(inside, view.shape, view.stride(), view.storage_offset()).fill_(True)
    return bool(torch.isnan(buf[~inside]).all())


def f64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def batch(tokens, vocab, g, idle=0.1):
    ids = torch.randint(0, vocab, (tokens,), generator=g, dtype=torch.int32)
    bad = torch.rand(tokens, generator=g) < idle
    wrong = torch.tensor([-1, vocab, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)
    return torch.where(bad, wrong[torch.arange(tokens) % 4], ids).cuda()


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("tokens,vocab,d,shift,pad", [(1, 1, 1, 0, 0), (5, 7, 3, 1, 2), (9, 100, 64, 0, 0), (33, 50, 257, 3, 1),
                                                      (700, 300, 4096, 0, 8), (4, 1000, 8192, 0, 0), (2049, 97, 36, 2, 2)])
@pytest.mark.parametrize("scale", [1.0, 2.5])
def test_lookup(spmv, dtype, tokens, vocab, d, shift, pad, scale):
    g = gen(tokens + d)
    table, _ = placed((torch.randn(vocab, d, generator=g) * 3).to(dtype), shift, pad)
    ids = batch(tokens, vocab, g)
    out, buf = placed(torch.zeros(tokens, d, dtype=dtype), pad, shift)
    got = spmv.embed_rows(table, ids, scale=scale, out=out)
    assert got is out and untouched(out, buf)
    want = ref.embed(f64(table), ids.tolist(), scale)
    if scale == 1.0:
        assert np.array_equal(f64(got), want)
    else:
        assert np.all(np.abs(f64(got) - want) <= (H[dtype] + 2 * E) * np.abs(want) + TINY[dtype])
    assert torch.equal(spmv.embed_rows(table, ids, scale=scale), got)


def test_lookup_keeps_bits(spmv):
    """NaN payloads, infinities and -0 of a row that is only copied; 0 for padding beside a table of NaN."""
    bits = torch.randint(-2 ** 15, 2 ** 15, (64, 72), generator=gen(1), dtype=torch.int16).cuda()
    ids = torch.tensor([3, -1, 63, 0], dtype=torch.int32).cuda()
    got = spmv.embed_rows(bits.view(torch.bfloat16), ids).view(torch.int16)
    assert torch.equal(got[[0, 2, 3]], bits[[3, 63, 0]]) and not got[1].any()
    nan = torch.full((4, 8), math.nan, device="cuda")
    assert not spmv.embed_rows(nan, torch.full((5,), -1, dtype=torch.int32, device="cuda"), scale=math.inf).any()


def check_grad(spmv, ids, dx, vocab, scale, out_dtype, out=None, accumulate=False):
    base = f64(out) if accumulate else 0.0
    got = spmv.embed_rows_grad(dx, ids, vocab, scale=scale, out=out, accumulate=accumulate, dtype=out_dtype)
    want, mag, count = ref.embed_grad(f64(dx), ids.tolist(), vocab, scale)
    err = (count[:, None] + 2) * E * mag
    want = want + base
    err = err + (H[out_dtype] + (E if accumulate else 0)) * (np.abs(want) + err) + TINY[out_dtype]
    assert np.all(np.abs(f64(got) - want) <= err)
    if not accumulate:
        assert not f64(got)[count == 0].any()
    return got


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("tokens,vocab,d", [(1, 1, 1), (3, 5, 7), (31, 4, 8), (33, 2, 40), (500, 40, 129), (1000, 3, 20),
                                            (5000, 700, 24), (9000, 4, 16), (20000, 513, 8), (40000, 70000, 4), (70001, 100001, 3)])
@pytest.mark.parametrize("wide", [False, True])
def test_gradient(spmv, dtype, tokens, vocab, d, wide):
    g = gen(tokens + vocab)
    ids, dx = batch(tokens, vocab, g), torch.randn(tokens, d, generator=g).to(dtype).cuda()
    out = torch.float32 if wide else dtype
    first = check_grad(spmv, ids, dx, vocab, 1.0, out)
    again = check_grad(spmv, ids, dx, vocab, -0.75, out, out=first.clone(), accumulate=True)
    assert torch.equal(spmv.embed_rows_grad(dx, ids, vocab, dtype=out), first)  # the same bits every time
    rest = torch.ones(vocab, dtype=torch.bool)
    there = ids.cpu()
    rest[there[(there >= 0) & (there < vocab)].long()] = False
    assert torch.equal(again[rest.cuda()], first[rest.cuda()])


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("shift,pad", [(1, 0), (3, 5), (0, 8), (2, 2), (4, 4)])
@pytest.mark.parametrize("d", [1, 24, 100, 515])
def test_gradient_any_address(spmv, dtype, shift, pad, d):
    g = gen(d + pad)
    ids = batch(300, 37, g)
    dx, _ = placed(torch.randn(300, d, generator=g).to(dtype), shift, pad)
    for out_dtype in {dtype, torch.float32}:
        out, buf = placed(torch.randn(37, d, generator=g).to(out_dtype), pad, shift)
        check_grad(spmv, ids, dx, 37, 1.5, out_dtype, out=out)
        check_grad(spmv, ids, dx, 37, 1.5, out_dtype, out=out, accumulate=True)
        assert untouched(out, buf)


@pytest.mark.parametrize("tokens", [1, 32, 33, 64, 1000, 4097, 40000])
@pytest.mark.parametrize("d", [8, 300])
def test_gradient_of_one_row(spmv, tokens, d):
    """every token the same: the row's sum is joined from all shares"""
    dx = torch.randn(tokens, d, generator=gen(tokens)).cuda()
    check_grad(spmv, torch.full((tokens,), 5, dtype=torch.int32, device="cuda"), dx, 9, 1.0, torch.float32)


def test_gradient_of_runs(spmv):
    """rows that begin or end with a share, cover exactly one, or several"""
    counts = [32, 32, 1, 31, 64, 7, 25, 96, 16, 16, 33, 31, 300, 20]
    ids = torch.repeat_interleave(torch.arange(len(counts), dtype=torch.int32), torch.tensor(counts))
    ids = ids[torch.randperm(len(ids), generator=gen(3))].cuda()
    dx = torch.randn(len(ids), 40, generator=gen(4)).cuda()
    check_grad(spmv, ids, dx, len(counts) + 2, 1.0, torch.float32)


@pytest.mark.parametrize("vocab", [2, 512, 513, 262144, 262145, 2 ** 21])
def test_gradient_digits(spmv, vocab):
    """one digit, two and three, at the borders between them"""
    ids = torch.tensor([vocab - 1, 0, vocab - 1, vocab // 2, vocab, 1 % vocab, vocab - 2], dtype=torch.int32).cuda()
    check_grad(spmv, ids, torch.randn(7, 4, generator=gen(5)).cuda(), vocab, 1.0, torch.float32)


def test_gradient_exact_on_integers(spmv):
    g = gen(6)
    ids = batch(3000, 50, g)
    dx = torch.randint(-4, 5, (3000, 16), generator=g).float().cuda()
    want, _, _ = ref.embed_grad(f64(dx), ids.tolist(), 50, 1.0)
    assert np.array_equal(f64(spmv.embed_rows_grad(dx, ids, 50)), want)


def test_no_tokens(spmv):
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    dx = torch.empty(0, 5, device="cuda")
    assert spmv.embed_rows(torch.ones(4, 5, device="cuda"), none).shape == (0, 5)
    assert not spmv.embed_rows_grad(dx, none, 4).any()
    out = torch.ones(4, 5, device="cuda")
    assert spmv.embed_rows_grad(dx, none, 4, out=out, accumulate=True).eq(1).all()
    pad = torch.full((40,), -1, dtype=torch.int32, device="cuda")
    assert not spmv.embed_rows_grad(torch.full((40, 5), math.nan, device="cuda"), pad, 4).any()


def test_lookup_and_gradient_against_differences(spmv):
    """<dx, embed(table + h v) - embed(table)> / h = <embed_grad(dx), v>: both are linear"""
    g = gen(7)
    table, v = torch.randn(60, 33, generator=g).cuda(), torch.randn(60, 33, generator=g).cuda()
    ids, dx = batch(200, 60, g), torch.randn(200, 33, generator=g).cuda()
    ahead, here = spmv.embed_rows(table + v, ids, scale=3.0), spmv.embed_rows(table, ids, scale=3.0)
    by_steps = float((dx.double() * (ahead.double() - here.double())).sum())
    by_grad = float((spmv.embed_rows_grad(dx, ids, 60, scale=3.0).double() * v.double()).sum())
    terms = float((dx.abs().double() * (ahead.abs() + here.abs()).double()).sum())
    assert abs(by_steps - by_grad) <= 16 * E * terms


def test_streams_and_graph(spmv):
    g = gen(8)
    table = torch.randn(500, 64, generator=g).cuda().bfloat16()
    ids, dx = batch(6000, 500, g), torch.randn(6000, 64, generator=g).cuda().bfloat16()
    want, want_grad = spmv.embed_rows(table, ids, scale=2.0), spmv.embed_rows_grad(dx, ids, 500)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x, grad = spmv.embed_rows(table, ids, scale=2.0, stream=side), spmv.embed_rows_grad(dx, ids, 500, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(x, want) and torch.equal(grad, want_grad)
    static_ids, static_dx = torch.zeros_like(ids), torch.zeros_like(dx)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x = spmv.embed_rows(table, static_ids, scale=2.0)
        grad = spmv.embed_rows_grad(static_dx, static_ids, 500)
    for seed in (1, 2):
        static_ids.copy_(batch(6000, 500, gen(seed)))
        static_dx.copy_(dx * seed)
        graph.replay()
        assert torch.equal(x, spmv.embed_rows(table, static_ids, scale=2.0))
        assert torch.equal(grad, spmv.embed_rows_grad(static_dx, static_ids, 500))


def test_far_rows(spmv):
    """offsets beyond 2^31 values, on both sides"""
    vocab, d = 70000, 33000  # 2.3e9 values
    table = torch.zeros(vocab, d, dtype=torch.bfloat16, device="cuda")
    table[-1] = 3.0
    ids = torch.tensor([vocab - 1, 0, vocab - 2, vocab - 1], dtype=torch.int32, device="cuda")
    assert spmv.embed_rows(table, ids).float().sum(1).tolist() == [3.0 * d, 0, 0, 3.0 * d]
    dx = torch.ones(4, d, dtype=torch.bfloat16, device="cuda")
    spmv.embed_rows_grad(dx, ids, vocab, out=table)
    assert float(table[-1].float().mean()) == 2.0 and float(table[-2].float().mean()) == 1.0
    assert float(table[0].float().mean()) == 1.0 and not table[1:-2].any()
