"""The gradient of the table lookup where its sort has nothing to do, and from a host thread of its own."""
import math
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spmv():
    import __graft_entry__

    __graft_entry__._build_module().build()
    import sparse_matrix_vector_csr_gb300 as spmv

    return spmv


@pytest.mark.parametrize("vocab", [300, 513, 262145])
@pytest.mark.parametrize("tokens", [1, 40, 3000])
def test_gradient_without_a_token(spmv, vocab, tokens):
    """batches of padding alone, with rows of one digit, two and three: the later passes of the sort have nothing"""
    ids = torch.full((tokens,), -1, dtype=torch.int32)
    ids[::3] = vocab
    dx = torch.full((tokens, 5), math.nan, device="cuda")
    assert not spmv.embed_rows_grad(dx, ids.cuda(), vocab).any()
    out = torch.ones(vocab, 5, device="cuda")
    assert spmv.embed_rows_grad(dx, ids.cuda(), vocab, out=out, accumulate=True).eq(1).all()


def test_first_call_of_a_host_thread(spmv):
    """a host thread that has made no CUDA call yet: the library's is the first"""
    from sparse_matrix_vector_csr_gb300._abi import _check, lib

    table, ids = torch.randn(600, 24, generator=torch.Generator().manual_seed(1)).cuda(), torch.arange(0, 700, 7, dtype=torch.int32).cuda()
    want = spmv.embed_rows(table, ids)
    want_grad = spmv.embed_rows_grad(want, ids, 600)
    x, grad = torch.zeros_like(want), torch.ones_like(table)
    n = spmv.spmv_embed_workspace(100, 600, 24)
    space = torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    failed = []

    def work(entry, args):
        try:
            _check(entry(*args))
        except spmv.SpmvError as e:
            failed.append(str(e))

    for entry, args in ((lib.spmv_embed_rows, (100, 600, 24, ids.data_ptr(), table.data_ptr(), 24, 1.0, x.data_ptr(), 24, 1, None)),
                        (lib.spmv_embed_rows_grad, (100, 600, 24, ids.data_ptr(), want.data_ptr(), 24, 1, 1.0, 0, grad.data_ptr(), 24, 1,
                                                    space.data_ptr(), n, None))):
        t = threading.Thread(target=work, args=(entry, args))
        t.start()
        t.join()
    assert not failed, failed
    torch.cuda.synchronize()
    assert torch.equal(x, want) and torch.equal(grad, want_grad)
