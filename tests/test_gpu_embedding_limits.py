"""Tables of nearly 2^31 rows, the most that an embedding is created for."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
MOST = 2**31 - 2


@pytest.mark.parametrize("back", [0, 13, 14, 15, 100, 1300])
def test_gradient_of_the_tallest_tables(back):
    """Rows that only an earlier call named are zero again; few tokens and none take their own launches."""
    from powersgd_rank_gradient_gb300 import Embedding

    vocab = MOST - back
    e = Embedding(vocab, 1, 3000, device=DEV)
    dw = torch.full((vocab, 1), 5.0, dtype=torch.float16, device=DEV)
    flat = dw[:, 0]
    # the first and last rows, and some around every power of two on the way
    rows = torch.cat([torch.arange(6), torch.tensor([2**k + d for k in range(8, 31) for d in (-1, 0, 3)]),
                      vocab - 1 - torch.arange(6)]).to(DEV)
    assert int(rows.max()) < vocab and rows.unique().numel() == rows.numel()
    for tokens, pick in ((3000, rows), (3000, rows[:40:3]), (10, rows), (2000, rows[:3]), (0, rows)):
        ids = pick[torch.arange(tokens, device=DEV) % pick.numel()]
        e.backward(ids, torch.ones((tokens, 1), dtype=torch.float16, device=DEV), out=dw)
        found, count = ids.unique(return_counts=True)
        got = flat[found].clone()
        assert torch.equal(got, count.to(torch.float16))  # whole numbers below 2048: exact
        flat[found] = 0
        assert not any(bool(part.any()) for part in flat.split(2**28)), "a row that no token names is not zero"
        flat[found] = got  # what the next call has to clear
    assert not e.status()
