"""Two host threads with handles and streams of their own."""

import threading

import pytest

import training_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("dim", [64, 65])
def test_handles_of_two_threads(dim):
    from powersgd_rank_gradient_gb300 import Embedding, LayerNorm, distill_loss

    done = {}

    def work(seed):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        with torch.cuda.stream(torch.cuda.Stream()):
            e, n = Embedding(3000, dim, 5000, device=DEV), LayerNorm(dim, device=DEV)
            ids = torch.randint(0, 3000, (5000,), device=DEV, generator=gen)
            g = torch.empty((5000, dim), device=DEV).normal_(0, 1, generator=gen)
            results = []
            for _ in range(20):
                y, mean, rstd = n.forward(g)
                results.append((e.backward(ids, g), y, *n.backward(g, g, mean, rstd), *distill_loss(y, g[:, :9], (ids[:, None] + torch.arange(9, device=DEV)) % dim)))
            for r in results[1:]:
                assert all(torch.equal(a, b) for a, b in zip(r, results[0]))
            dw, mag, count = tu.table_grad(ids, g, 3000, 1.0)
            tu.check(results[0][0], dw, tu.table_grad_tol(dw, mag, count, torch.float32))
            want, err = tu.norm_backward(g, g, mean, rstd, None)
            for a, b, c in zip(results[0][2:5], want, err):
                tu.check(a, b, tu.out_tol(c, b, torch.float32))
            done[seed] = True

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert done == {0: True, 1: True}
