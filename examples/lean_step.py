"""Data-parallel language-model training that keeps little, on one GPU.

One residual block (RMS norm, feed-forward layer) between an embedding and an
output layer tied to it, in bf16 with fp32 parameters.  Between the forward and
the backward pass a step keeps 8-bit checkpoints of what the norms and the
feed-forward layer's products read, and no logits at all.  Every replica's
gradients are written straight into its flat fp32 bucket -- the table's by the
output layer and then, accumulated, by the embedding -- and ``powerSGD_hook``
averages the buckets compressed.

    python examples/lean_step.py [--steps 40] [--replicas 2] [--rank 8]
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from powersgd_rank_gradient_gb300 import (Embedding, LinearCrossEntropy, LinearWeightGrad, PowerSGDState, RMSNorm,  # noqa: E402
                                          powerSGD_hook, save_activation)

PAD = 0
NO_TARGET = -100


class Model:
    """Parameters in one flat fp32 buffer, laid out as the gradient buckets are."""

    def __init__(self, vocab, dim, hidden, tokens, device="cuda", seed=0):
        self.shapes = [(vocab, dim), (dim,), (hidden, dim), (dim, hidden), (dim,)]
        self.numel = sum(math.prod(s) for s in self.shapes)
        gen = torch.Generator(device=device).manual_seed(seed)
        self.params = torch.zeros(self.numel, device=device)
        table, w1, up, down, w2 = self.views(self.params)
        table.normal_(0, dim ** -0.5, generator=gen)
        up.normal_(0, dim ** -0.5, generator=gen)
        down.normal_(0, hidden ** -0.5, generator=gen)
        w1.fill_(1.0)
        w2.fill_(1.0)
        self.embedding = Embedding(vocab, dim, tokens, padding_idx=PAD, scale=math.sqrt(dim), device=device)
        self.norm1, self.norm2 = RMSNorm(dim, device=device), RMSNorm(dim, device=device)
        self.up_grad = LinearWeightGrad(hidden, dim, tokens, device=device)
        self.down_grad = LinearWeightGrad(dim, hidden, tokens, device=device)
        self.loss = LinearCrossEntropy(vocab, dim, tokens, device=device)

    def views(self, flat):
        """The tensors of a flat bucket, in bucket order."""
        out, at = [], 0
        for s in self.shapes:
            n = math.prod(s)
            out.append(flat[at:at + n].view(s))
            at += n
        return out

    def gradients(self, ids, targets, bucket):
        """Writes the gradients of the mean loss over the tokens that have a target into
        ``bucket``; returns that loss."""
        table, w1, up, down, w2 = (p.bfloat16() for p in self.views(self.params))
        g_table, g_w1, g_up, g_down, g_w2 = self.views(bucket)
        live = (targets >= 0).float()
        weights = live / live.sum()
        # forward: the feed-forward layer reads the norm's output as the checkpoint holds it
        x = self.embedding.forward(table, ids)
        kept_y, _, rstd1 = self.norm1.forward8(x, w1)
        kept_x = save_activation(x)
        act = torch.nn.functional.gelu(kept_y.restore(torch.bfloat16) @ up.t())
        kept_act = save_activation(act)
        z, summed, rstd2 = self.norm2.forward(act @ down.t(), w2, residual=x)
        kept_sum = save_activation(summed)
        losses, lse = self.loss.forward(z, table, targets, weights)
        del x, act, summed
        # backward
        dz, _ = self.loss.backward(z, table, targets, lse, weights, dweight=g_table)
        dsum, _ = self.norm2.backward(dz, kept_sum, rstd2, w2, dweight=g_w2)
        self.down_grad.backward(dsum, kept_act, out=g_down)
        pre = (kept_y.restore(torch.bfloat16) @ up.t()).requires_grad_()
        (dpre,) = torch.autograd.grad(torch.nn.functional.gelu(pre), pre, dsum @ down)
        self.up_grad.backward(dpre, kept_y, out=g_up)
        dx, _ = self.norm1.backward(dpre @ up, kept_x, rstd1, w1, grad_summed=dsum, dweight=g_w1)
        self.embedding.backward(ids, dx, out=g_table, accumulate=True)
        return losses.sum()

    def status(self):
        """Raises if an operator reported a failure since the last status."""
        assert not self.embedding.status()
        for op in (self.up_grad, self.down_grad, self.loss):
            op.status()


def batch(gen, sequences, length, following, device):
    """Token ids with padded ends, and what follows each by a fixed rule (no target for padding)."""
    vocab = following.shape[0]
    ids = torch.randint(1, vocab, (sequences, length), device=device, generator=gen)
    ends = torch.randint(length // 2, length + 1, (sequences, 1), device=device, generator=gen)
    ids = torch.where(torch.arange(length, device=device) < ends, ids, PAD)
    return ids, torch.where(ids != PAD, following[ids], NO_TARGET)


def train(steps=40, replicas=2, rank=8, vocab=509, dim=256, hidden=512, sequences=8, length=64, rate=1.0, device="cuda", seed=0):
    """Runs ``steps`` steps; returns the losses."""
    model = Model(vocab, dim, hidden, sequences * length, device, seed)
    state = PowerSGDState(model.shapes, replicas, matrix_approximation_rank=rank, start_powerSGD_iter=2, device=device)
    buckets = [torch.empty(model.numel, device=device) for _ in range(replicas)]
    gen = torch.Generator(device=device).manual_seed(seed + 1)
    following = torch.randint(1, vocab, (vocab,), device=device, generator=gen)
    history = []
    for _ in range(steps):
        loss = 0.0
        for bucket in buckets:
            loss = loss + model.gradients(*batch(gen, sequences, length, following, device), bucket) / replicas
        model.params.add_(powerSGD_hook(state, buckets), alpha=-rate)
        history.append(loss)
    model.status()
    assert not state.status()
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
