"""Data-parallel distillation with compressed gradients, on one GPU.

A small student language model (embedding, layer norm, one linear layer, layer
norm, an output layer tied to the embedding) learns from a teacher's top logits.
Every replica's gradients are written straight into its flat bucket by the
training operators -- the table's by the output layer and then, accumulated, by
the embedding -- and ``powerSGD_hook`` averages the buckets compressed.

    python examples/distill_step.py [--steps 40] [--replicas 2] [--rank 8]
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from powersgd_rank_gradient_gb300 import Embedding, LayerNorm, PowerSGDState, distill_loss, powerSGD_hook  # noqa: E402

PAD = 0


class Student:
    """Parameters in one flat fp32 buffer, laid out as the gradient buckets are."""

    def __init__(self, vocab, dim, tokens, device="cuda", seed=0):
        self.shapes = [(vocab, dim), (dim,), (dim,), (dim, dim), (dim,), (dim,)]
        self.numel = sum(math.prod(s) for s in self.shapes)
        gen = torch.Generator(device=device).manual_seed(seed)
        self.params = torch.zeros(self.numel, device=device)
        table, w1, _, linear, w2, _ = self.views(self.params)
        table.normal_(0, dim ** -0.5, generator=gen)
        linear.normal_(0, dim ** -0.5, generator=gen)
        w1.fill_(1.0)
        w2.fill_(1.0)
        self.embedding = Embedding(vocab, dim, tokens, padding_idx=PAD, scale=math.sqrt(dim), device=device)
        self.norm1, self.norm2 = LayerNorm(dim, device=device), LayerNorm(dim, device=device)

    def views(self, flat):
        """The tensors of a flat bucket, in bucket order."""
        out, at = [], 0
        for s in self.shapes:
            n = math.prod(s)
            out.append(flat[at:at + n].view(s))
            at += n
        return out

    def gradients(self, ids, teacher_logits, teacher_indices, temperature, bucket):
        """Writes the gradients of the mean loss over the tokens that are not
        padding into ``bucket``; returns that loss."""
        table, w1, b1, linear, w2, b2 = self.views(self.params)
        g_table, g_w1, g_b1, g_linear, g_w2, g_b2 = self.views(bucket)
        dim = table.shape[1]
        live = (ids != PAD).float()
        weights = live / live.sum()
        # forward
        x = self.embedding.forward(table, ids)
        y, mean1, rstd1 = self.norm1.forward(x, w1, b1)
        h = torch.nn.functional.gelu(y @ linear.t())
        z, mean2, rstd2 = self.norm2.forward(h, w2, b2)
        logits = z @ table.t()
        # loss and its gradient, in the logits' own memory
        losses, dlogits = distill_loss(logits, teacher_logits, teacher_indices, temperature, weights, dlogits=logits)
        # backward
        flat = dlogits.view(-1, table.shape[0])
        torch.mm(flat.t(), z.view(-1, dim), out=g_table)
        dz = (flat @ table).view_as(z)
        dh, _, _ = self.norm2.backward(dz, h, mean2, rstd2, w2, dweight=g_w2, dbias=g_b2)
        pre = (y @ linear.t()).requires_grad_()
        (dpre,) = torch.autograd.grad(torch.nn.functional.gelu(pre), pre, dh)
        torch.mm(dpre.view(-1, dim).t(), y.view(-1, dim), out=g_linear)
        dx, _, _ = self.norm1.backward(dpre @ linear, x, mean1, rstd1, w1, dweight=g_w1, dbias=g_b1)
        self.embedding.backward(ids, dx, out=g_table, accumulate=True)
        return losses.sum()


def batch(gen, sequences, length, vocab, device):
    """Token ids with padded ends."""
    ids = torch.randint(1, vocab, (sequences, length), device=device, generator=gen)
    ends = torch.randint(length // 2, length + 1, (sequences, 1), device=device, generator=gen)
    return torch.where(torch.arange(length, device=device) < ends, ids, PAD)


def train(steps=40, replicas=2, rank=8, vocab=509, dim=256, sequences=8, length=64, k=16, temperature=2.0, rate=1.0,
          device="cuda", seed=0):
    """Runs ``steps`` steps; returns the losses."""
    student = Student(vocab, dim, sequences * length, device, seed)
    state = PowerSGDState(student.shapes, replicas, matrix_approximation_rank=rank, start_powerSGD_iter=2, device=device)
    buckets = [torch.empty(student.numel, device=device) for _ in range(replicas)]
    gen = torch.Generator(device=device).manual_seed(seed + 1)
    # the teacher: a fixed distribution after each token
    teacher = torch.empty((vocab, vocab), device=device).normal_(0, 3, generator=gen)
    history = []
    for _ in range(steps):
        loss = 0.0
        for bucket in buckets:
            ids = batch(gen, sequences, length, vocab, device)
            top, at = teacher[ids].topk(k, dim=-1)
            loss = loss + student.gradients(ids, top, at, temperature, bucket) / replicas
        mean = powerSGD_hook(state, buckets)
        student.params.add_(mean, alpha=-rate)
        history.append(loss)
    assert not student.embedding.status() and not state.status()
    return [float(x) for x in history]


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--steps", type=int, default=40)
    p.add_argument("--replicas", type=int, default=2)
    p.add_argument("--rank", type=int, default=8)
    a = p.parse_args()
    for i, loss in enumerate(train(a.steps, a.replicas, a.rank)):
        if i % 5 == 0 or i + 1 == a.steps:
            print(f"step {i:4d}  loss {loss:.4f}")


if __name__ == "__main__":
    main()
