"""Lookups into outputs of other orders than the tokens'."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def setup(dim, batch, seq, seed=0):
    from powersgd_rank_gradient_gb300 import Embedding

    gen = torch.Generator(device=DEV).manual_seed(seed)
    weight = torch.empty((50, dim), device=DEV).normal_(0, 1, generator=gen)
    ids = torch.randint(0, 50, (batch, seq), device=DEV, generator=gen)
    return Embedding(50, dim, batch * seq, device=DEV), weight, ids


@pytest.mark.parametrize("dim", [1, 7, 24, 300])
@pytest.mark.parametrize("batch,seq", [(5, 7), (1, 6), (6, 1), (2, 33)])
@pytest.mark.parametrize("gap", [0, 3, 8])
def test_sequence_first_output(dim, batch, seq, gap):
    """Batch-first ids into a buffer whose rows lie sequence first, with and without room between them."""
    e, weight, ids = setup(dim, batch, seq)
    room = torch.full((seq, batch, dim + gap), 9.0, device=DEV)
    out = room[:, :, :dim].transpose(0, 1)
    assert e.forward(weight, ids, out=out) is out
    assert torch.equal(out, weight[ids])
    assert bool((room[:, :, dim:] == 9.0).all())


def test_overlapping_rows_are_refused():
    from powersgd_rank_gradient_gb300._lib import PsgdError

    e, weight, ids = setup(8, 3, 4)
    room = torch.zeros(400, device=DEV)
    for strides in ((0, 8), (8, 0), (7, 24), (32, 7), (8, 23), (31, 8), (8, 8)):
        with pytest.raises(PsgdError, match="rows overlap"):
            e.forward(weight, ids, out=room.as_strided((3, 4, 8), strides + (1,)))
    for strides in ((8, 24), (32, 8), (9, 26), (33, 8)):
        out = room.as_strided((3, 4, 8), strides + (1,))
        assert torch.equal(e.forward(weight, ids, out=out), weight[ids])
