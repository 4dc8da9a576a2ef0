"""The operators that keep a step small, together: one step's bucket against 64-bit arithmetic, captured and replayed,
on another stream, and the example."""

import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import step_util as su  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
DEV = "cuda:0"


def values(x):
    """What x is in 8 bits."""
    v, s = su.eight(x, su.E4)
    return v * su.spread(s, x.shape[-1])


def reference(model, ids, targets, pad):
    """(loss, gradients) of the step in 64 bits, from the same bf16 parameters, with the checkpoints' roundings."""
    table, w1, up, down, w2 = (p.bfloat16().double() for p in model.views(model.params))
    dim = table.shape[1]
    flat, t = ids.flatten(), targets.flatten()
    live = t >= 0
    x = table[flat] * math.sqrt(dim)
    (y, r1), _ = su.rms_forward(x, w1, model.norm1.eps)
    y8 = values(y)
    pre = (y8 @ up.t()).requires_grad_()
    act = torch.nn.functional.gelu(pre)
    s = x + act.detach() @ down.t()
    (z, r2), _ = su.rms_forward(s, w2, model.norm2.eps)
    logits = (z @ table.t()).requires_grad_()
    loss = torch.nn.functional.cross_entropy(logits[live], t[live])
    (g,) = torch.autograd.grad(loss, logits)
    g_table = g.t() @ z
    (ds, g_w2), _ = su.rms_backward(g @ table, values(s), r2, w2)
    g_down = ds.t() @ values(act.detach())
    (dpre,) = torch.autograd.grad(act, pre, ds @ down)
    g_up = dpre.t() @ y8
    (dx, g_w1), _ = su.rms_backward(dpre @ up, values(x), r1, w1, ds)
    keep = flat != pad
    g_table = g_table.index_add(0, flat[keep], dx[keep] * math.sqrt(dim))
    return loss.detach(), [g_table, g_w1, g_up, g_down, g_w2]


@pytest.mark.parametrize("vocab,dim,hidden,length", [(301, 64, 136, 17), (1003, 136, 200, 40), (700, 256, 512, 64)])
def test_step_against_64_bits(vocab, dim, hidden, length):
    import lean_step as ex

    model = ex.Model(vocab, dim, hidden, 4 * length, DEV, seed=3)
    gen = torch.Generator(device=DEV).manual_seed(5)
    following = torch.randint(1, vocab, (vocab,), device=DEV, generator=gen)
    ids, targets = ex.batch(gen, 4, length, following, DEV)
    bucket = torch.full((model.numel,), float("nan"), device=DEV)
    loss = model.gradients(ids, targets, bucket)
    model.status()
    want_loss, want = reference(model, ids, targets, ex.PAD)
    # bf16 between the operators: some ten roundings of 2^-8 at most, 2^-10 on average, on a path; and a value whose
    # rounding crosses a border of its 8-bit format is a step of 2^-3 off, which 2^-8 / 2^-3 of the values do: 2^-3 * 2^-2.5 of the
    # norm at most
    assert abs(float(loss) - float(want_loss)) <= 10 * 2.0 ** -8 * abs(float(want_loss))
    for got, exp in zip(model.views(bucket), want):
        assert float((got.double() - exp).norm()) <= (2.0 ** -5.5 + 10 * 2.0 ** -9) * float(exp.norm())


def test_a_step_captured_and_on_another_stream():
    import lean_step as ex

    model = ex.Model(509, 128, 256, 512, DEV, seed=1)
    gen = torch.Generator(device=DEV).manual_seed(2)
    following = torch.randint(1, 509, (509,), device=DEV, generator=gen)
    ids, targets = ex.batch(gen, 8, 64, following, DEV)
    buckets = [torch.zeros(model.numel, device=DEV) for _ in range(3)]
    model.gradients(ids, targets, buckets[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        model.gradients(ids, targets, buckets[1])
    side.synchronize()
    assert torch.equal(buckets[0], buckets[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loss = model.gradients(ids, targets, buckets[2])
    graph.replay()
    assert torch.equal(buckets[0], buckets[2]) and math.isfinite(float(loss))
    other, more = ex.batch(gen, 8, 64, following, DEV)
    ids.copy_(other), targets.copy_(more)
    graph.replay()
    model.gradients(ids, targets, buckets[0])
    assert torch.equal(buckets[0], buckets[2])


def test_example_runs():
    import lean_step as ex

    assert all(math.isfinite(x) for x in ex.train(steps=12, device=DEV))
