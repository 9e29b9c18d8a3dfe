"""Train a small layer of sparse experts on a teacher's top logits.

A student (embedding, router, experts, output matrix) learns a random teacher's distribution over a
vocabulary of which only the k largest logits of each row, and their log-sum, are kept.  One step:

    teacher:  topk_rows             its logits -> k columns and values a row, log-sum
    student:  topk_rows             router logits -> experts and weights a token
              RoutePlan, dispatch   tokens sorted by expert
              (the experts' dense products, by torch)
              combine               experts' rows back to tokens, weighted
              distill_loss_grad     loss, and its gradient in place of the logits
              combine_grad, dispatch_grad, TopRows.grad   back to the experts, the tokens, the router

    python examples/distill_sparse_experts.py [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_matrix_vector_csr_gb300 as spmv  # noqa: E402


class Student:
    """Token -> embedding + sum over its experts of weight * (row @ U_e) -> logits."""

    def __init__(self, tokens, d, experts, k, vocab, align, generator):
        def matrix(*shape, scale):
            return torch.randn(*shape, generator=generator, device="cuda") * scale

        self.experts, self.k, self.align = experts, k, align
        self.weights = {"embed": matrix(tokens, d, scale=1.0), "router": matrix(d, experts, scale=d ** -0.5),
                        "up": matrix(experts, d, d, scale=d ** -0.5), "out": matrix(d, vocab, scale=d ** -0.5)}
        self.velocity = {n: torch.zeros_like(w) for n, w in self.weights.items()}

    def products(self, rows, offsets, weights):
        """Every segment's rows times its expert's matrix (the segments' ends come to the host)."""
        out = torch.zeros(rows.shape[0], weights.shape[2], device=rows.device)
        for e in range(self.experts):
            out[offsets[e]:offsets[e + 1]] = rows[offsets[e]:offsets[e + 1]] @ weights[e]
        return out

    def step(self, token, target, lr):
        w = self.weights
        x = w["embed"][token]
        top = spmv.topk_rows(x @ w["router"], self.k, weights="selected")
        plan = spmv.RoutePlan(top.ids, self.experts, align=self.align)
        offsets = plan.offsets.tolist()
        xs = plan.dispatch(x)
        ys = self.products(xs, offsets, w["up"])
        h = x + plan.combine(ys, top.weights)
        z = h @ w["out"]
        loss, dz = spmv.distill_loss_grad(z, target.ids, target.vals, teacher_lse=target.lse, scale=1.0 / len(token),
                                          out=z)
        dh = dz @ w["out"].t()
        dys, dweights = plan.combine_grad(dh, ys, top.weights)
        dxs = self.products(dys, offsets, w["up"].transpose(1, 2))
        dlogits = top.grad(dweights)
        dx = dh + plan.dispatch_grad(dxs) + dlogits @ w["router"].t()
        grads = {"out": h.t() @ dz, "router": x.t() @ dlogits, "up": torch.zeros_like(w["up"]),
                 "embed": torch.zeros_like(w["embed"]).index_add_(0, token, dx)}
        for e in range(self.experts):
            a, b = offsets[e], offsets[e + 1]
            grads["up"][e] = xs[a:b].t() @ dys[a:b]
        for n, g in grads.items():
            self.velocity[n].mul_(0.9).add_(g)
            w[n].sub_(self.velocity[n], alpha=lr)
        return loss, grads


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=512, help="different tokens, all in each batch")
    ap.add_argument("--d", type=int, default=128)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--k", type=int, default=2, help="experts a token")
    ap.add_argument("--vocab", type=int, default=5000)
    ap.add_argument("--kept", type=int, default=32, help="teacher logits kept a row")
    ap.add_argument("--lr", type=float, default=4.0)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    teacher_logits = torch.randn(a.tokens, a.vocab, generator=g, device="cuda") * 2.0
    target = spmv.topk_rows(teacher_logits, a.kept, lse=True)
    student = Student(a.tokens, a.d, a.experts, a.k, a.vocab, 16, g)
    token = torch.arange(a.tokens, device="cuda")
    losses = []
    for i in range(a.steps):
        loss, _ = student.step(token, target, a.lr)
        losses.append(float(loss.mean()))
        if i % 10 == 0 or i == a.steps - 1:
            print(f"step {i:4d}  mean loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    main()
