"""The gradient of the table lookup where its sort has nothing to do."""
import math

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
