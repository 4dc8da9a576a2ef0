"""Cross entropy of a linear layer without its logits against its 64-bit definition."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import step_util as su  # noqa: E402

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def randn(shape, dtype, seed, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0, std, generator=g)


def handle(vocab, dim, tokens):
    from powersgd_rank_gradient_gb300 import LinearCrossEntropy

    return LinearCrossEntropy(vocab, dim, tokens, device=DEV)


def batch(tokens, vocab, dim, dtype, seed, masked=0.25, known=6.0):
    """hidden, weight, targets: some targets known to the model, some outside the vocabulary."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    weight = randn((vocab, dim), dtype, seed + 1, dim ** -0.5)
    t = torch.randint(0, vocab, (tokens,), device=DEV, generator=gen)
    hidden = (randn((tokens, dim), F32, seed + 2) + known * torch.rand((tokens, 1), device=DEV, generator=gen) * weight[t].float()).to(dtype)
    out = torch.rand(tokens, device=DEV, generator=gen) < masked
    return hidden, weight, torch.where(out, torch.tensor([-100, vocab, -1, 2**31 - 1], device=DEV)[t % 4], t)


def run(h, hidden, weight, targets, weights=None, scale=1.0, odtype=F32, accumulate=False, seed=0):
    losses, lse = h.forward(hidden, weight, targets, weights)
    (wl, ws), (el, es) = su.loss_forward(hidden, weight, targets, weights)
    su.check(losses, wl, el)
    su.check(lse, ws, es)
    v, d = weight.shape
    bucket = torch.full((v * d + 9,), 7.0, dtype=odtype, device=DEV)
    dw = bucket[3:3 + v * d].view(v, d)
    before = randn((v, d), odtype, seed + 9, 0.01) if accumulate else None
    if accumulate:
        dw.copy_(before)
    dh, gw = h.backward(hidden, weight, targets, lse, weights, grad_scale=scale, dweight=dw, accumulate=accumulate)
    h.status()
    assert gw is dw and dh.shape == hidden.shape and dh.dtype == hidden.dtype
    (wh, ww), (eh, ew) = su.loss_backward(hidden, weight, targets, lse, weights, scale, before)
    su.check_out(dh, wh, eh, hidden.dtype)
    su.check_out(dw, ww, ew, odtype)
    assert bool((bucket[:3] == 7.0).all()) and bool((bucket[3 + v * d:] == 7.0).all())
    first = bucket.clone()
    if accumulate:
        dw.copy_(before)
    again = h.forward(hidden, weight, targets, weights)
    dh2, _ = h.backward(hidden, weight, targets, lse, weights, grad_scale=scale, dweight=dw, accumulate=accumulate)
    assert torch.equal(again[0], losses) and torch.equal(again[1], lse), "another result from the same inputs"
    assert torch.equal(dh, dh2) and torch.equal(first, bucket), "another result from the same inputs"
    return losses, lse, dh, first[3:3 + v * d].view(v, d)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens,vocab,dim", [(256, 256, 64), (1, 256, 64), (1, 1, 1), (3, 7, 5), (130, 300, 72), (257, 1000, 100),
                                              (64, 5000, 256), (1000, 777, 33), (500, 2049, 1601)])
def test_sizes(tokens, vocab, dim, dtype):
    run(handle(vocab, dim, tokens), *batch(tokens, vocab, dim, dtype, tokens + vocab + dim))


@pytest.mark.parametrize("dtype,odtype", [(BF16, F32), (BF16, BF16), (BF16, F16), (F16, F32), (F16, F16), (F16, BF16)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_types(dtype, odtype, accumulate):
    hidden, weight, targets = batch(200, 600, 136, dtype, 5)
    run(handle(600, 136, 200), hidden, weight, targets.to(torch.int32), scale=1024.0 if odtype == F16 else 1.0, odtype=odtype,
        accumulate=accumulate)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("kind", ["mean", "unequal", "far apart", "negative", "some zero"])
def test_weights(dtype, kind):
    hidden, weight, targets = batch(300, 500, 64, dtype, 7)
    g = torch.Generator(device=DEV).manual_seed(3)
    w = {"mean": torch.full((300,), 1 / 300, device=DEV), "unequal": 0.01 + torch.rand(300, device=DEV, generator=g),
         "far apart": torch.exp2(torch.randint(-20, 20, (300,), device=DEV, generator=g).float()),
         "negative": torch.randn(300, device=DEV, generator=g),
         "some zero": torch.randint(0, 3, (300,), device=DEV, generator=g).float()}[kind]
    run(handle(500, 64, 300), hidden, weight, targets, w, scale=256.0)


@pytest.mark.parametrize("offset", [0, 1])
def test_a_vocabulary_in_pieces(offset):
    """8192 tokens: 16384 columns of the logits' gradient at a time."""
    hidden, weight, targets = batch(8192, 34000, 72, BF16, 11, masked=0.1)
    flat = torch.zeros(weight.numel() + offset, dtype=BF16, device=DEV)
    placed = flat[offset:].view(34000, 72)
    placed.copy_(weight)
    h = handle(34000, 72, 8192)
    assert h.workspace_bytes() < 8192 * 34000 * 2
    run(h, hidden, placed, targets, torch.full((8192,), 1 / 8192, device=DEV), accumulate=offset == 1)


def test_few_tokens_and_a_long_vocabulary():
    run(handle(50257, 200, 5), *batch(5, 50257, 200, BF16, 13, masked=0.0))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens,vocab,dim", [(1, 50257, 1600), (2, 1001, 8), (3, 4099, 328), (4, 130, 8192), (4, 5000, 8200), (1, 3, 64)])
def test_tokens_one_by_one(tokens, vocab, dim, dtype):
    """Four tokens at most, with and without rows that are read whole."""
    hidden, weight, targets = batch(tokens, vocab, dim, dtype, 71, masked=0.0)
    h = handle(vocab, dim, 300)
    run(h, hidden, weight, targets)
    targets[tokens // 2] = -100
    run(h, hidden, weight, targets)
    hidden[0], weight[vocab // 2, 3] = torch.nan, torch.inf
    losses, _ = h.forward(hidden, weight, targets)
    # (an infinite weight's logit is -infinity, which has no mass, where the hidden value is negative)
    z, live = hidden.double() @ weight.double().t(), targets >= 0
    bad = torch.isnan(z).any(1) | (z == torch.inf).any(1)
    assert torch.equal(~torch.isfinite(losses[live]), bad[live]) and not bool(losses[~live].any())


def test_sums_that_are_cut():
    run(handle(300, 264, 5000), *batch(5000, 300, 264, F16, 17))


def test_layouts():
    h = handle(300, 72, 60)
    hidden, weight, targets = batch(60, 300, 72, BF16, 19)
    want = run(h, hidden, weight, targets)
    for offset, gap in [(0, 8), (1, 0), (8, 3)]:
        def place(x):
            flat = torch.zeros(offset + x.shape[0] * (72 + gap), dtype=BF16, device=DEV)
            view = flat[offset:].view(x.shape[0], 72 + gap)[:, :72]
            view.copy_(x)
            return view

        assert all(torch.equal(a, b) for a, b in zip(run(h, place(hidden), place(weight), targets), want))
        dh = torch.full((60, 72 + gap), 7.0, dtype=BF16, device=DEV)
        dw = torch.full((300, 72 + gap), 7.0, device=DEV)
        h.backward(hidden, weight, targets, want[1], dhidden=dh[:, :72], dweight=dw[:, gap:])
        assert torch.equal(dh[:, :72], want[2]) and torch.equal(dw[:, gap:], want[3])
        assert bool((dh[:, 72:] == 7).all()) and bool((dw[:, :gap] == 7).all())
    shaped = run(h, hidden.view(3, 4, 5, 72), weight, targets.view(3, 4, 5))
    assert all(torch.equal(a.flatten(), b.flatten()) for a, b in zip(shaped, want))
    one = run(h, hidden[7], weight, torch.tensor(5, device=DEV))
    assert one[0].shape == () and one[2].shape == (72,)
    run(h, hidden[:1].expand(60, 72), weight, targets)
    run(h, hidden, weight[:1].expand(300, 72), targets)


def test_padding_costs_nothing_and_touches_nothing():
    """Tokens that do not count may hold anything; the others' results are those of a batch without them, bit for bit."""
    hidden, weight, targets = batch(700, 900, 80, BF16, 23, masked=0.5)
    w = torch.rand(700, device=DEV) + 0.1
    w[::7] = 0
    h = handle(900, 80, 700)
    keep = (targets >= 0) & (targets < 900) & (w != 0)
    want = run(h, hidden[keep], weight, targets[keep], w[keep])
    hidden[~keep] = torch.nan
    losses, lse, dh, dw = run(h, hidden, weight, targets, w)
    assert torch.equal(losses[keep], want[0]) and torch.equal(lse[keep], want[1])
    assert torch.equal(dh[keep], want[2]) and torch.equal(dw, want[3])
    assert not bool(losses[~keep].any()) and not bool(lse[~keep].any()) and not bool(dh[~keep].any())


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens", [0, 5, 300])
def test_no_token_counts(tokens, accumulate):
    h = handle(1000, 64, 300)
    run(h, *batch(300, 1000, 64, BF16, 29))  # leaves its own behind
    hidden, weight, targets = batch(tokens, 1000, 64, BF16, 31, masked=1.0)
    _, _, dh, dw = run(h, hidden, weight, targets, accumulate=accumulate)
    assert not bool(dh.any()) and (accumulate or not bool(dw.any()))


def test_calls_of_many_sizes_on_one_handle():
    h = handle(700, 136, 3000)
    for tokens in (3000, 1, 257, 256, 255, 2999, 0, 64):
        run(h, *batch(tokens, 700, 136, F16, tokens))


def test_large_logits():
    for size, dtype in [(300.0, BF16), (3e3, F16)]:
        hidden, weight, targets = batch(100, 500, 64, dtype, 37)
        hidden *= size
        losses, lse = handle(500, 64, 100).forward(hidden, weight, targets)
        (wl, ws), (el, es) = su.loss_forward(hidden, weight, targets, None)
        su.check(losses, wl, el)
        su.check(lse, ws, es)


def test_nan_and_infinity_stay_in_their_rows():
    hidden, weight, targets = batch(300, 500, 64, BF16, 41, masked=0.0)
    h = handle(500, 64, 300)
    losses, lse = h.forward(hidden, weight, targets)
    dh, _ = h.backward(hidden, weight, targets, lse)
    hidden[5, 3], hidden[270, 1] = torch.nan, torch.inf
    losses2, lse2 = h.forward(hidden, weight, targets)
    dh2, dw2 = h.backward(hidden, weight, targets, lse2)
    keep = torch.ones(300, dtype=torch.bool, device=DEV)
    keep[[5, 270]] = False
    assert torch.equal(losses2[keep], losses[keep]) and torch.equal(lse2[keep], lse[keep]) and torch.equal(dh2[keep], dh[keep])
    assert bool(torch.isnan(losses2[~keep]).all()) and bool(torch.isnan(dh2[~keep]).all()) and bool(torch.isnan(dw2).any())


def test_gradient_against_differences():
    """Both gradients against central differences of the forward definition in 64 bits."""
    hidden, weight, targets = batch(40, 90, 48, BF16, 43)
    w = torch.rand(40, device=DEV)
    h = handle(90, 48, 40)
    _, lse = h.forward(hidden, weight, targets, w)
    dh, dw = h.backward(hidden, weight, targets, lse, w)

    def loss(x, y):
        return float(su.loss_forward(x, y, targets, w)[0][0].sum())

    eps = 1e-4
    for k in range(5):
        a, b = randn((40, 48), F32, 50 + k).double(), randn((90, 48), F32, 60 + k).double()
        x, y = hidden.double(), weight.double()
        slope = (loss(x + eps * a, y + eps * b) - loss(x - eps * a, y - eps * b)) / (2 * eps)
        got = float((dh.double() * a).sum() + (dw.double() * b).sum())
        # G is rounded to bf16 and dh again, 2^-8 of each term at most
        size = float((dh.double() * a).abs().sum() + (dw.double() * b).abs().sum())
        assert abs(got - slope) <= 2 * 2.0 ** -8 * size


def test_streams_and_graphs():
    hidden, weight, targets = batch(600, 3000, 128, BF16, 47)
    h = handle(3000, 128, 600)

    def step(**kw):
        losses, lse = h.forward(hidden, weight, targets, **kw)
        return (losses, lse, *h.backward(hidden, weight, targets, lse, **kw))

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    h.status(stream=side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.cuda.graph(other):
        got2 = step()
    for g, out in ((graph, got), (other, got2), (graph, got)):
        hidden2, _, targets2 = batch(600, 3000, 128, BF16, 48)
        hidden.copy_(hidden2), targets.copy_(targets2)
        g.replay()
        fresh = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(fresh, step()))
    before = got[3]._version
    h.backward(hidden, weight, targets, got[1], dweight=got[3])
    assert got[3]._version == before + 1


def test_refusals():
    from powersgd_rank_gradient_gb300._lib import PsgdError

    hidden, weight, targets = batch(20, 50, 64, BF16, 53)
    h = handle(50, 64, 20)
    losses, lse = h.forward(hidden, weight, targets)
    for call, words in [
        (lambda: h.forward(hidden.float(), weight, targets), "hidden must be float16 or bfloat16"),
        (lambda: h.forward(hidden, weight.half(), targets), "weight must have hidden's type"),
        (lambda: h.forward(hidden, weight[:49], targets), "weight must be"),
        (lambda: h.forward(hidden, weight.t().contiguous().t(), targets), "contiguous in its last"),
        (lambda: h.forward(hidden, weight, targets[:19]), "targets must be a contiguous"),
        (lambda: h.forward(hidden, weight, targets.float()), "targets must be int32 or int64"),
        (lambda: h.forward(hidden, weight, targets, losses.double()), "weights must be a contiguous float32"),
        (lambda: h.forward(hidden, weight, targets, losses.cpu()), "weights must be on cuda"),
        (lambda: h.forward(hidden.cpu(), weight, targets), "must be on cuda"),
        (lambda: h.backward(hidden, weight, targets, lse[:19]), "lse must be"),
        (lambda: h.backward(hidden, weight, targets, lse, dhidden=hidden.float()), "dhidden must have"),
        (lambda: h.backward(hidden, weight, targets, lse, dweight=weight[:49]), "dweight must be"),
        (lambda: h.backward(hidden, weight, targets, lse, accumulate=True), "accumulate needs"),
        (lambda: h.forward(hidden.clone().requires_grad_(), weight, targets), "hidden requires a gradient"),
        (lambda: h.forward(hidden, weight.clone().requires_grad_(), targets), "weight requires a gradient"),
    ]:
        with pytest.raises(ValueError, match=words):
            call()
    for call in [lambda: h.backward(hidden, weight, targets, lse, dhidden=hidden), lambda: h.backward(hidden, weight, targets, lse, dweight=weight)]:
        with pytest.raises(PsgdError, match="overlap"):
            call()
    with pytest.raises(PsgdError, match="max_tokens"):
        h.forward(torch.cat([hidden, hidden]), weight, torch.cat([targets, targets]))
    h.close()
    with pytest.raises(PsgdError, match="NULL"):
        h.forward(hidden, weight, targets)
