"""Operators of a training step that keeps little between its forward and its
backward pass, as cases to measure.

Root-mean-square norm with the residual's addition (output in the input's type or
in 8 bits with scales; its backward pass, which may read an 8-bit checkpoint),
activation checkpoints in 8 bits (saving, restoring, and the weight gradient of
a linear layer from one), and the softmax cross entropy of a linear output layer
without its logits (losses, and the gradients of both operands).

``run`` computes a case in plain torch operations in 32 bits (64 where values lie
next to a rounding border) while ``own`` is false, and with this package's entry
points while it is true.  ``exact`` states the definitions in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
          "e5m2": torch.float8_e5m2}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
BLOCK = 128  # elements of a row that share a scale in 8 bits
# an 8-bit format: its largest value is LIMIT * 2^TOP, its values' significands have BITS bits behind the
# leading one, and below 2^LOW they are equally spaced
LIMIT = 0.875
TOP = {"e4m3": 9, "e5m2": 16}
BITS = {"e4m3": 3, "e5m2": 2}
LOW = {"e4m3": -6, "e5m2": -14}


# -- cases ---------------------------------------------------------------------

def _norm(name, op, rows, dim, xtype, ptype, residual=True, saved="none"):
    return {"name": name, "op": op, "rows": rows, "dim": dim, "xtype": xtype, "ptype": ptype, "residual": residual,
            "saved": saved}


def _save(name, rows, dim, xtype, otype, saved):
    return {"name": name, "op": "save", "rows": rows, "dim": dim, "xtype": xtype, "otype": otype, "saved": saved}


def _wgrad(name, rows, outs, ins, gtype, otype, saved, offset=0):
    return {"name": name, "op": "wgrad", "rows": rows, "outs": outs, "ins": ins, "gtype": gtype, "otype": otype,
            "saved": saved, "offset": offset}


def _loss(name, op, rows, vocab, dim, xtype, idtype="i64", pad=0.0, offset=0, weighted=False):
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "dim": dim, "xtype": xtype, "idtype": idtype,
            "pad": pad, "offset": offset, "weighted": weighted, "scale": 65536.0 if xtype == "f16" else 1.0}


def listed():
    return [
        # one row of GPT-2-XL's width, as a decoding step normalises it: latency
        _norm("rms_one_row", "rms", 1, 1600, "bf16", "bf16"),
        # GPT-2-XL's activations of 32 sequences of 1024, the residual added in the same pass
        _norm("rms_gpt2_xl", "rms", 32768, 1600, "bf16", "bf16"),
        # BERT-large's activations of 32 sequences of 512, the output kept in 8 bits for the backward pass and restored there
        _norm("rms_8bit_bert_large", "rms8", 16384, 1024, "bf16", "f32", saved="e4m3"),
        # rows of odd length in a count that divides into nothing; the sum was kept as it is
        _norm("rms_backward_odd", "rmsbwd", 4099, 1023, "f16", "f32"),
        # GPT-2-XL's activations of 64 sequences of 1024, the sum kept in 8 bits
        _norm("rms_backward_gpt2_xl_8bit", "rmsbwd", 65536, 1600, "bf16", "bf16", saved="e4m3"),
        # BERT-large's widest activations, saved after the forward pass and restored in the backward pass
        _save("checkpoint_bert_large", 16384, 4096, "bf16", "bf16", "e4m3"),
        # one sequence's weight gradient of an attention projection of BERT-large, fp32 bucket at an odd place
        _wgrad("wgrad_bert_large_attention", 509, 1024, 1024, "f16", "f32", "e4m3", offset=3),
        # GPT-2-XL's first feed-forward matrix, 16 sequences of 1024
        _wgrad("wgrad_gpt2_xl_ffn", 16384, 6400, 1600, "bf16", "f32", "e4m3"),
        # one token scored over GPT-2-XL's vocabulary: the table is read once
        _loss("loss_one_token", "loss", 1, 50257, 1600, "bf16"),
        # BERT-large's masked tokens (15 % of 32 x 512) and their losses
        _loss("loss_bert_large", "loss", 2458, 30522, 1024, "f16", idtype="i32"),
        # the gradients of one padded sequence of 499 tokens over BERT-large's table, into a bucket at an odd place
        _loss("loss_backward_bert_large", "lossbwd", 499, 30522, 1024, "bf16", pad=0.4, offset=5),
        # 8 sequences of 1024 over GPT-2-XL's vocabulary, ends padded
        _loss("loss_backward_gpt2_xl", "lossbwd", 8192, 50257, 1600, "bf16", pad=0.25),
    ]


MOST_BYTES = 0.7e9  # of a drawn case that moves data; the largest listed one moves 0.74e9
MOST_FLOPS = 2.5e12  # of a drawn case that multiplies; the largest listed one does 3.5e12


def _spread(rng, low, high):
    """A whole number, uniform in its logarithm."""
    return min(max(int(round(math.exp(rng.uniform(math.log(low), math.log(high))))), low), high)


def _width(rng, high=6400):
    """A model width: mostly a multiple of 64, now and then any number."""
    d = _spread(rng, 64, high)
    return max(64, d // 64 * 64) if rng.random() < 0.7 else d


def _drawn(rng):
    op = rng.choice(["rms", "rms8", "rmsbwd", "save", "wgrad", "loss", "lossbwd"])
    x = rng.choice(["f32", "f16", "bf16"])
    half = rng.choice(["f16", "bf16"])
    saved = rng.choice(["e4m3", "e4m3", "e5m2"])
    if op in ("rms", "rms8", "rmsbwd"):
        if op == "rms" or (op == "rmsbwd" and rng.random() < 0.5):
            saved = "none"
        x = half if op == "rms8" else x
        return _norm("", op, _spread(rng, 1, 65536), _width(rng), x, rng.choice(["f32", x]), rng.random() < 0.7, saved)
    if op == "save":
        return _save("", _spread(rng, 1, 65536), _width(rng), x, half, saved)
    if op == "wgrad":
        return _wgrad("", _spread(rng, 1, 32768), _width(rng), _width(rng), half, rng.choice(["f32", half]), saved,
                      rng.choice([0, 0, 1, 4, 1023]))
    return _loss("", op, _spread(rng, 1, 8192), _spread(rng, 1000, 50257), _width(rng, 1600), half, rng.choice(["i32", "i64"]),
                 rng.choice([0.0, 0.25, 0.5]), rng.choice([0, 0, 1, 4, 1023]), rng.random() < 0.3)


def draw(rng):
    while True:
        case = _drawn(rng)
        w = work(case)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS:
            del case["name"]
            return case


# -- inputs --------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(gen, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _activations(gen, rows, dim, dtype):
    """Activations: some channels much larger than the others, as trained models have them."""
    x = _randn(gen, (rows, dim), torch.float32)
    channel = torch.exp(_randn(gen, (dim,), torch.float32, 0.7))
    return (x * channel).to(dtype)


def _blocks(x):
    """(rows, blocks, BLOCK), the last block of a row filled up with zeros."""
    n = -(-x.shape[1] // BLOCK)
    return torch.nn.functional.pad(x, (0, n * BLOCK - x.shape[1])).view(x.shape[0], n, BLOCK)


def _to_8bit(x, saved):
    """(codes, scales): a block's scale is the least power of two that brings its largest value within the format."""
    x = x if x.dtype == torch.float64 else x.float()
    b = _blocks(x)
    part, exponent = torch.frexp(b.abs().amax(2))
    exponent = (exponent - TOP[saved] + (part > LIMIT).int()).clamp(min=-126)
    scales = torch.where(part > 0, torch.ldexp(torch.ones_like(part), exponent), 1.0).float()
    codes = (b / scales[:, :, None]).view(x.shape[0], -1)[:, :x.shape[1]]
    if x.dtype == torch.float64:  # one rounding: straight to the format's step
        least = torch.frexp(codes.abs())[1].sub_(1).clamp_(min=LOW[saved])
        step = torch.ldexp(torch.ones_like(codes), least - BITS[saved])
        codes = torch.round(codes / step) * step
    return codes.float().to(DTYPES[saved]).contiguous(), scales


def _values(codes, scales):
    """What 8-bit codes and their scales stand for."""
    return (_blocks(codes.float()) * scales[:, :, None]).view(codes.shape[0], -1)[:, :codes.shape[1]]


def _inputs(case, seed):
    gen, c, op = _generator(seed), case, case["op"]
    st = {"case": c}
    if op in ("rms", "rms8", "rmsbwd"):
        x, p, n, d = DTYPES[c["xtype"]], DTYPES[c["ptype"]], c["rows"], c["dim"]
        st["x"] = _activations(gen, n, d, x)
        st["weight"] = _randn(gen, (d,), p, 0.1).add_(1.0)
        st["residual"] = _randn(gen, (n, d), x, 2.0) if c["residual"] else None
        if op == "rmsbwd":
            st["grad"] = _randn(gen, (n, d), x)
            # the residual's own gradient, where the sum goes on past the norm
            st["grad_summed"], st["residual"] = st["residual"], None
            if c["saved"] != "none":
                st["codes"], st["scales"] = _to_8bit(st["x"], c["saved"])
            xd = st["x"].float()
            st["rstd"] = torch.rsqrt((xd * xd).mean(1) + EPS)
    elif op == "save":
        st["x"] = _activations(gen, c["rows"], c["dim"], DTYPES[c["xtype"]])
    elif op == "wgrad":
        st["codes"], st["scales"] = _to_8bit(_activations(gen, c["rows"], c["ins"], DTYPES[c["gtype"]]), c["saved"])
        st["grad"] = _randn(gen, (c["rows"], c["outs"]), DTYPES[c["gtype"]], 0.05)
    else:
        n, v, d, x = c["rows"], c["vocab"], c["dim"], DTYPES[c["xtype"]]
        st["weight"] = _randn(gen, (v, d), x, d ** -0.5)
        target = torch.randint(0, v, (n,), device="cuda", generator=gen)
        # a model that has learned some of its targets, others not
        known = torch.rand((n, 1), device="cuda", generator=gen) * 14.0
        st["hidden"] = (torch.randn((n, d), device="cuda", generator=gen) + known * st["weight"][target].float()).to(x)
        live = torch.rand(n, device="cuda", generator=gen) >= c["pad"]
        st["targets"] = torch.where(live, target, -100).to(torch.int32 if c["idtype"] == "i32" else torch.int64)
        # the mean over the tokens, or tokens of unequal weight
        st["weights"] = torch.full((n,), 1.0 / n, device="cuda")
        if c["weighted"]:
            st["weights"] *= 0.1 + 2.0 * torch.rand(n, device="cuda", generator=gen)
        if op == "lossbwd":
            st["lse"] = torch.zeros(n, device="cuda")
            for lo in range(0, n, 2048):
                z = st["hidden"][lo:lo + 2048].float() @ st["weight"].float().t()
                top = z.amax(1)
                st["lse"][lo:lo + 2048] = top + torch.log(torch.exp(z - top[:, None]).sum(1))
            st["lse"] = torch.where(live, st["lse"], 0.0)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    op, c = case["op"], case
    # the buffers a training program keeps: the bucket that gradients of parameters are written into
    if op == "rmsbwd":
        st["weight_grad"] = torch.empty(c["dim"], dtype=DTYPES[c["ptype"]], device="cuda")
    elif op in ("wgrad", "lossbwd"):
        shape = (c["outs"], c["ins"]) if op == "wgrad" else (c["vocab"], c["dim"])
        bucket = torch.empty(c["offset"] + shape[0] * shape[1], device="cuda",
                             dtype=DTYPES[c["otype"] if op == "wgrad" else c["xtype"]])
        st["weight_grad"] = bucket[c["offset"]:].view(shape)
    if own:
        import powersgd_rank_gradient_gb300 as psgd

        if "codes" in st:
            st["saved"] = psgd.Activation8(st["codes"], st["scales"])
        if op in ("rms", "rms8", "rmsbwd"):
            st["op"] = psgd.RMSNorm(c["dim"], eps=EPS)
        elif op == "save":
            st["op"] = psgd.save_activation
        elif op == "wgrad":
            st["op"] = psgd.LinearWeightGrad(c["outs"], c["ins"], max_tokens=c["rows"])
        else:
            st["op"] = psgd.LinearCrossEntropy(c["vocab"], c["dim"], max_tokens=c["rows"])
    return st


# -- one pass ------------------------------------------------------------------

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    c, op = st["case"], st["op"]
    kind = c["op"]
    if kind == "rms":
        return op.forward(st["x"], st["weight"], st["residual"])
    if kind == "rms8":
        saved, summed, rstd = op.forward8(st["x"], st["weight"], st["residual"], dtype=DTYPES[c["saved"]])
        return saved.restore(DTYPES[c["xtype"]]), summed, rstd
    if kind == "rmsbwd":
        return op.backward(st["grad"], st["x"] if c["saved"] == "none" else st["saved"], st["rstd"], st["weight"],
                           grad_summed=st["grad_summed"], dweight=st["weight_grad"])
    if kind == "save":
        saved = op(st["x"], dtype=DTYPES[c["saved"]])
        return saved.restore(DTYPES[c["otype"]]), saved.scales
    if kind == "wgrad":
        return op.backward(st["grad"], st["saved"], out=st["weight_grad"])
    if kind == "loss":
        return op.forward(st["hidden"], st["weight"], st["targets"], weights=st["weights"])
    return op.backward(st["hidden"], st["weight"], st["targets"], st["lse"], weights=st["weights"],
                       grad_scale=c["scale"], dweight=st["weight_grad"])


def _run_plain(st):
    c = st["case"]
    kind = c["op"]
    if kind in ("rms", "rms8"):
        s = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).to(st["x"].dtype)
        f = s.double() if kind == "rms8" else s.float()
        rstd = torch.rsqrt((f * f).mean(1) + EPS)
        y = f * rstd[:, None] * st["weight"].to(f.dtype)
        y = y if kind == "rms" else _values(*_to_8bit(y, c["saved"]))
        return y.to(s.dtype), s, rstd.float()
    if kind == "rmsbwd":
        x = st["x"].float() if c["saved"] == "none" else _values(st["codes"], st["scales"])
        g, xh = st["grad"].float(), x * st["rstd"][:, None]
        a = g * st["weight"].float()
        dx = st["rstd"][:, None] * (a - xh * (a * xh).mean(1, keepdim=True))
        if st["grad_summed"] is not None:
            dx = dx + st["grad_summed"].float()
        return dx.to(st["grad"].dtype), (g * xh).sum(0).to(DTYPES[c["ptype"]])
    if kind == "save":
        codes, scales = _to_8bit(st["x"], c["saved"])
        return _values(codes, scales).to(DTYPES[c["otype"]]), scales
    if kind == "wgrad":
        return (st["grad"].float().t() @ _values(st["codes"], st["scales"])).to(DTYPES[c["otype"]])
    h, w, t, loss_weight = st["hidden"].float(), st["weight"].float(), st["targets"].long(), st["weights"]
    live = (t >= 0) & (t < c["vocab"]) & (loss_weight != 0)
    at = torch.where(live, t, 0)[:, None]
    z = h @ w.t()
    if kind == "loss":
        top = z.amax(1, keepdim=True)
        lse = (top + torch.log(torch.exp(z - top).sum(1, keepdim=True)))[:, 0]
        return torch.where(live, loss_weight * (lse - z.gather(1, at)[:, 0]), 0.0), torch.where(live, lse, 0.0)
    q = torch.exp(z - st["lse"][:, None])
    q = q.scatter_add_(1, at, torch.full_like(q[:, :1], -1.0))
    q = torch.where(live[:, None], q * (loss_weight * c["scale"])[:, None], 0.0)
    return (q @ w).to(st["hidden"].dtype), (q.t() @ h).to(DTYPES[c["xtype"]])


# -- the definitions in 64 bits --------------------------------------------------

def _nearest(v, saved):
    """The value of an 8-bit format (within its range) next to each v, ties to the even one."""
    binade = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** LOW[saved])))
    step = torch.exp2(binade - BITS[saved])
    return torch.round(v / step) * step


def _exact_8bit(x, saved):
    """(values, scales) of x in 8 bits: block by block along the row."""
    most = LIMIT * 2.0 ** TOP[saved]
    values, scales = torch.empty_like(x), []
    for lo in range(0, x.shape[1], BLOCK):
        b = x[:, lo:lo + BLOCK]
        top = b.abs().max(1).values
        scale = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, 1.0) / most)).clamp(min=-126))
        scale = torch.where(top > scale * most, 2 * scale, scale)
        scale = torch.where(top > 0, scale, 1.0)
        values[:, lo:lo + BLOCK] = _nearest(b / scale[:, None], saved) * scale[:, None]
        scales.append(scale)
    return values, torch.stack(scales, 1)


def exact(case, seed):
    st, c = _inputs(case, seed), case
    op = c["op"]
    if op in ("rms", "rms8"):
        s = st["x"].double()
        if st["residual"] is not None:
            s = (s + st["residual"].double()).to(st["x"].dtype).double()
        rstd = (torch.einsum("ij,ij->i", s, s) / c["dim"] + EPS) ** -0.5
        y = torch.einsum("ij,i,j->ij", s, rstd, st["weight"].double())
        return (y if op == "rms" else _exact_8bit(y, c["saved"])[0]), s, rstd
    if op == "rmsbwd":
        # the sums of a row and of a column as products, dx from them
        x = st["x"].double() if c["saved"] == "none" else _exact_8bit(st["x"].double(), c["saved"])[0]
        g, r, w = st["grad"].double(), st["rstd"].double(), st["weight"].double()
        dw = torch.einsum("ij,ij,i->j", g, x, r)
        along = torch.einsum("ij,ij,j->i", g, x, w) * r ** 3 / c["dim"]
        dx = torch.einsum("ij,i,j->ij", g, r, w) - x * along[:, None]
        return (dx if st["grad_summed"] is None else dx + st["grad_summed"].double()), dw
    if op == "save":
        return _exact_8bit(st["x"].double(), c["saved"])
    if op == "wgrad":
        x = torch.cat([b * s[:, None] for b, s in zip(st["codes"].float().double().split(BLOCK, 1),
                                                      st["scales"].double().unbind(1))], 1)
        return torch.einsum("ti,tj->ij", st["grad"].double(), x)
    n, w = c["rows"], st["weight"].double()
    losses, lses = torch.zeros(n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
    dh = torch.zeros((n, c["dim"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros_like(w)
    for lo in range(0, n, 2048):  # rows are independent but for the table's gradient, which adds up
        hi = min(n, lo + 2048)
        t, lw = st["targets"][lo:hi].long(), st["weights"][lo:hi].double()
        live = ((t >= 0) & (t < c["vocab"]) & (lw != 0)).nonzero()[:, 0]
        h, t, lw = st["hidden"][lo:hi].double()[live], t[live], lw[live]
        z = torch.einsum("td,vd->tv", h, w)
        if op == "loss":
            lse = torch.logsumexp(z, 1)
            lses[lo + live] = lse
            losses[lo + live] = lw * (lse - z[torch.arange(len(t), device="cuda"), t])
            continue
        q = torch.exp(z - st["lse"][lo:hi].double()[live][:, None])
        q[torch.arange(len(t), device="cuda"), t] -= 1.0
        q *= c["scale"] * lw[:, None]
        dh[lo + live] = torch.einsum("tv,vd->td", q, w)
        dw += torch.einsum("tv,td->vd", q, h)
    return (losses, lses) if op == "loss" else (dh, dw)


# -- what a pass cannot do without -------------------------------------------------

def work(case):
    c, op = case, case["op"]
    if op in ("rms", "rms8", "rmsbwd"):
        n, d, b, p = c["rows"], c["dim"], SIZE[c["xtype"]], SIZE[c["ptype"]]
        code = 1.0 + 4.0 / BLOCK
        if op == "rmsbwd":
            # gradient, what was kept and (with a residual) the gradient of the sum read, one gradient and the weight's written
            kept = b if c["saved"] == "none" else code
            return {"bytes": n * d * (2 * b + kept + (b if c["residual"] else 0)) + 4 * n + 2 * d * p, "flops": 11 * n * d}
        # x read, y written; with a residual that is read and the sum written.  The 8-bit form leaves its codes besides
        return {"bytes": n * d * (b * (4 if c["residual"] else 2) + (code if op == "rms8" else 0)) + 4 * n + d * p,
                "flops": n * d * (5 if op == "rms" else 9)}
    if op == "save":
        n = c["rows"] * c["dim"]
        return {"bytes": n * (SIZE[c["xtype"]] + SIZE[c["otype"]] + 1 + 4 / BLOCK), "flops": 4 * n}
    if op == "wgrad":
        n, i, o = c["rows"], c["ins"], c["outs"]
        return {"bytes": n * o * SIZE[c["gtype"]] + n * i * (1 + 4 / BLOCK) + i * o * SIZE[c["otype"]], "flops": 2 * n * i * o}
    # rows that count, both operands read once; the gradients of both written once.  Logits are not among the backward
    # pass's inputs: it cannot do without their product
    n, v, d, b = c["rows"], c["vocab"], c["dim"], SIZE[c["xtype"]]
    live = n * (1.0 - c["pad"])
    ids = n * (4 + (4 if c["idtype"] == "i32" else 8))
    if op == "loss":
        return {"bytes": live * d * b + v * d * b + ids + 8 * n, "flops": 2 * live * v * d + 4 * live * v}
    return {"bytes": 2 * v * d * b + (live + n) * d * b + ids + 4 * n, "flops": 6 * live * v * d + 4 * live * v}
