"""The distillation example runs, learns, and its step's gradients are those of the same step under
autograd (float32 on both sides: the two differ by rounding only)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__

    __graft_entry__._build_module().build()
    spec = importlib.util.spec_from_file_location("distill_example",
                                                  os.path.join(ROOT, "examples", "distill_sparse_experts.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_learns(example):
    losses = example.main(["--steps", "40", "--tokens", "200", "--vocab", "1111", "--d", "64"])
    assert losses[-1] < 0.5 * losses[0]


def test_step_gradients_are_autograd_s(example):
    spmv = example.spmv
    g = torch.Generator(device="cuda").manual_seed(2)
    n, d, experts, k, vocab = 48, 32, 6, 2, 300
    student = example.Student(n, d, experts, k, vocab, 8, g)
    target = spmv.topk_rows(torch.randn(n, vocab, generator=g, device="cuda") * 2, 10, lse=True)
    token = torch.arange(n, device="cuda")
    w = {name: v.double().clone().requires_grad_() for name, v in student.weights.items()}
    x = w["embed"][token]
    val, ids = (x @ w["router"]).topk(k, dim=1)
    p = torch.softmax(val, 1)
    h = x + sum(p[:, j:j + 1] * torch.einsum("td,tdf->tf", x, w["up"][ids[:, j]]) for j in range(k))
    logq = torch.log_softmax(h @ w["out"], 1)
    t = target.ids.long()
    logp = target.vals.double() - target.lse.double()[:, None]
    rest = 1 - logp.exp().sum(1)
    others = torch.log(1 - logq.gather(1, t).exp().sum(1))
    loss = (logp.exp() * (logp - logq.gather(1, t))).sum(1) + rest * (rest.log() - others)
    loss.mean().backward()
    got, grads = student.step(token, target, 0.0)
    torch.testing.assert_close(got.double(), loss.detach(), rtol=1e-4, atol=1e-4)  # dense products in float32 (or tf32 off)
    for name, v in w.items():
        scale = v.grad.abs().max()
        assert (grads[name].double() - v.grad).abs().max() <= 1e-4 * scale, name
