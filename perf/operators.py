"""The training operators beside the gradient compressor, as cases to measure.

Three operators fill the buckets that the compressor takes: the embedding
(lookup with scaling, and the dense gradient of its table), layer norm (forward,
and backward with the reduction of its weight's and bias's gradients) and
distillation from a teacher's top logits (per-row losses and the logits'
gradient in one call).

``run`` computes a case in plain torch operations in 32 bits while ``own`` is
false, and with this package's entry points while it is true.  ``exact`` states
the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5


# -- cases ---------------------------------------------------------------------

def _lookup(name, vocab, dim, batch, seq, wtype, otype, idtype="i64", scale=1.0):
    return {"name": name, "op": "lookup", "vocab": vocab, "dim": dim, "batch": batch, "seq": seq, "wtype": wtype,
            "otype": otype, "idtype": idtype, "scale": scale}


def _embgrad(name, vocab, dim, batch, seq, gtype, otype, ids="text", idtype="i64", pad=False, offset=0, scale=1.0):
    return {"name": name, "op": "embgrad", "vocab": vocab, "dim": dim, "batch": batch, "seq": seq, "gtype": gtype,
            "otype": otype, "ids": ids, "idtype": idtype, "pad": pad, "offset": offset, "scale": scale}


def _norm(name, op, rows, dim, xtype, ptype):
    return {"name": name, "op": op, "rows": rows, "dim": dim, "xtype": xtype, "ptype": ptype}


def _distill(name, rows, vocab, k, ztype, ttype, temperature, masked=0.0, scale=1.0, idtype="i32", grad=True):
    return {"name": name, "op": "distill", "rows": rows, "vocab": vocab, "k": k, "ztype": ztype, "ttype": ttype,
            "temperature": temperature, "masked": masked, "scale": scale, "idtype": idtype, "grad": grad}


def listed():
    return [
        # one token of GPT-2-XL's table, as a decoding step looks it up: latency
        _lookup("lookup_one_token", 50257, 1600, 1, 1, "bf16", "bf16"),
        # BERT-large's input, 32 sequences of 512, fp32 table scaled by sqrt(dim)
        _lookup("lookup_bert_large", 30522, 1024, 32, 512, "f32", "f32", scale=32.0),
        # the gradient of that table into an fp32 bucket, sequences padded with id 0
        _embgrad("embgrad_bert_large", 30522, 1024, 32, 512, "f32", "f32", pad=True, scale=32.0),
        # GPT-2-XL's table, 16 sequences of 1024, 16-bit gradients in a 16-bit bucket
        _embgrad("embgrad_gpt2_xl", 50257, 1600, 16, 1024, "bf16", "bf16", idtype="i32"),
        # BERT-large's position table (every position once a sequence), 9 sequences of 499, at an odd place in its bucket
        _embgrad("embgrad_positions", 512, 1024, 9, 499, "f16", "f32", ids="position", offset=3),
        # one row of GPT-2-XL's width, as a decoding step normalises it: latency
        _norm("norm_one_row", "normfwd", 1, 1600, "bf16", "bf16"),
        # BERT-large's activations of 32 sequences of 512, parameters kept in fp32
        _norm("norm_bert_large", "normfwd", 16384, 1024, "bf16", "f32"),
        # rows of odd length, none of them aligned, in a count that divides into nothing
        _norm("norm_backward_odd", "normbwd", 4099, 1023, "f16", "f32"),
        # GPT-2-XL's activations of 64 sequences of 1024
        _norm("norm_backward_gpt2_xl", "normbwd", 65536, 1600, "bf16", "bf16"),
        # the next-token rows of five sequences over GPT-2-XL's vocabulary: few long rows
        _distill("distill_five_rows", 5, 50257, 16, "f32", "f32", 1.0),
        # BERT-large's masked tokens (15 % of 32 x 512), a tenth of them without a weight
        _distill("distill_bert_large", 2458, 30522, 32, "f32", "f16", 2.0, masked=0.1, idtype="i64"),
        # 8 sequences of 1024 over GPT-2-XL's vocabulary (rows of odd length), 16-bit logits
        _distill("distill_gpt2_xl", 8192, 50257, 64, "bf16", "bf16", 1.5, scale=1024.0),
    ]


MOST_BYTES = 1.4e9  # of a drawn case; the largest listed one moves 1.65e9


def _spread(rng, low, high):
    """A whole number, uniform in its logarithm (never 3072, which no configuration here has)."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    n = min(max(n, low), high)
    return n + 1 if n == 3072 else n


def _width(rng):
    """A model width: mostly a multiple of 64, now and then any number."""
    d = _spread(rng, 64, 6400)
    if rng.random() < 0.7:
        d = max(64, d // 64 * 64)
        d = 3136 if d == 3072 else d
    return d


def _drawn(rng):
    op = rng.choice(["lookup", "embgrad", "normfwd", "normbwd", "distill"])
    types = ["f32", "f16", "bf16"]
    if op == "lookup":
        return _lookup("", _spread(rng, 2, 50257), _width(rng), _spread(rng, 1, 64), _spread(rng, 1, 1024),
                       rng.choice(types), rng.choice(types), rng.choice(["i32", "i64"]), rng.choice([1.0, 32.0, 0.125]))
    if op == "embgrad":
        ids = "position" if rng.random() < 0.25 else "text"
        seq = _spread(rng, 1, 1024)
        vocab = max(seq, 2) if ids == "position" else _spread(rng, 2, 50257)
        g = rng.choice(types)
        return _embgrad("", vocab, _width(rng), _spread(rng, 1, 64), seq, g, rng.choice(["f32", g]), ids,
                        rng.choice(["i32", "i64"]), rng.random() < 0.5, rng.choice([0, 0, 1, 4, 1023]),
                        rng.choice([1.0, 32.0]))
    if op in ("normfwd", "normbwd"):
        x = rng.choice(types)
        return _norm("", op, _spread(rng, 1, 65536), _width(rng), x, rng.choice(["f32", x]))
    return _distill("", _spread(rng, 1, 8192), _spread(rng, 1000, 50257), rng.choice([1, 8, 32, 64, 100]), rng.choice(types),
                    rng.choice(types), rng.choice([1.0, 2.0, 4.0]), rng.choice([0.0, 0.2]), rng.choice([1.0, 1024.0]),
                    rng.choice(["i32", "i64"]), rng.random() < 0.75)


def draw(rng):
    while True:
        case = _drawn(rng)
        if work(case)["bytes"] <= MOST_BYTES:
            del case["name"]
            return case


# -- inputs --------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(gen, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _token_ids(c, gen):
    """(batch, seq) ids.  "text": ranks of a Zipf law (P(rank) ~ 1 / rank, as words have) over shuffled ids, the
    sequences' ends padded with id 0 where the case has padding.  "position": 0, 1, 2, ... in every sequence."""
    b, s, v = c["batch"], c["seq"], c["vocab"]
    dtype = torch.int32 if c["idtype"] == "i32" else torch.int64
    if c.get("ids", "text") == "position":
        return torch.arange(s, device="cuda").repeat(b, 1).to(dtype)
    u = torch.rand((b, s), device="cuda", generator=gen, dtype=torch.float64)
    rank = ((v + 1.0) ** u - 1.0).long().clamp_(0, v - 1)
    ids = torch.randperm(v, device="cuda", generator=gen)[rank]
    if c.get("pad"):
        length = torch.randint((s + 1) // 2, s + 1, (b, 1), device="cuda", generator=gen)
        ids = torch.where(torch.arange(s, device="cuda") < length, ids, 0)
    return ids.to(dtype)


def _inputs(case, seed):
    gen, c, op = _generator(seed), case, case["op"]
    st = {"case": c}
    if op == "lookup":
        st["ids"] = _token_ids(c, gen)
        st["weight"] = _randn(gen, (c["vocab"], c["dim"]), DTYPES[c["wtype"]], 0.02)
    elif op == "embgrad":
        st["ids"] = _token_ids(c, gen)
        st["grad"] = _randn(gen, (c["batch"], c["seq"], c["dim"]), DTYPES[c["gtype"]])
    elif op in ("normfwd", "normbwd"):
        x, p = DTYPES[c["xtype"]], DTYPES[c["ptype"]]
        st["x"] = _randn(gen, (c["rows"], c["dim"]), x, 1.5).add_(0.25)
        st["weight"] = _randn(gen, (c["dim"],), p, 0.1).add_(1.0)
        st["bias"] = _randn(gen, (c["dim"],), p, 0.1)
        if op == "normbwd":
            st["grad"] = _randn(gen, (c["rows"], c["dim"]), x)
            xd = st["x"].float()
            st["mean"] = xd.mean(1)
            st["rstd"] = torch.rsqrt((xd - st["mean"][:, None]).square().mean(1) + EPS)
    else:
        n, v, k = c["rows"], c["vocab"], c["k"]
        st["logits"] = _randn(gen, (n, v), DTYPES[c["ztype"]], 2.0)
        # the teacher's top logits, in descending order, at k different places of the row; the student has learned a part of them
        fall = torch.rand((n, k), device="cuda", generator=gen) * (8.0 / k)
        top = 12.0 - torch.cumsum(fall, 1)
        first = torch.randint(0, v, (n, 1), device="cuda", generator=gen)
        step = torch.randint(1, max(2, v // k), (n, 1), device="cuda", generator=gen)
        at = (first + step * torch.arange(k, device="cuda")) % v
        st["logits"].scatter_(1, at, (0.7 * top + torch.randn((n, k), device="cuda", generator=gen)).to(st["logits"].dtype))
        # ragged: a row keeps between one and all of its entries, the others are -1
        kept = torch.randint(1, k + 1, (n, 1), device="cuda", generator=gen)
        kept = torch.maximum(kept, torch.randint(1, k + 1, (n, 1), device="cuda", generator=gen))
        at = torch.where(torch.arange(k, device="cuda") < kept, at, -1)
        st["teacher"] = top.to(DTYPES[c["ttype"]])
        st["index"] = at.to(torch.int32 if c["idtype"] == "i32" else torch.int64)
        live = torch.rand(n, device="cuda", generator=gen) >= c["masked"]
        st["weights"] = live.float() / n
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    # the buffers a training program keeps: the bucket that gradients of parameters are written into
    if op == "embgrad":
        n = case["vocab"] * case["dim"]
        bucket = torch.empty(case["offset"] + n, dtype=DTYPES[case["otype"]], device="cuda")
        st["table_grad"] = bucket[case["offset"]:].view(case["vocab"], case["dim"])
    elif op == "normbwd":
        bucket = torch.empty(2 * case["dim"], dtype=DTYPES[case["ptype"]], device="cuda")
        st["weight_grad"], st["bias_grad"] = bucket[:case["dim"]], bucket[case["dim"]:]
    if own:
        import powersgd_rank_gradient_gb300 as psgd

        if op in ("lookup", "embgrad"):
            st["op"] = psgd.Embedding(case["vocab"], case["dim"], max_tokens=case["batch"] * case["seq"],
                                      padding_idx=0 if case.get("pad") else None, scale=case["scale"])
        elif op in ("normfwd", "normbwd"):
            st["op"] = psgd.LayerNorm(case["dim"], eps=EPS)
        else:
            st["op"] = psgd.distill_loss
    return st


# -- one pass ------------------------------------------------------------------

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    c, op = st["case"], st["op"]
    kind = c["op"]
    if kind == "lookup":
        return op.forward(st["weight"], st["ids"], out_dtype=DTYPES[c["otype"]])
    if kind == "embgrad":
        return op.backward(st["ids"], st["grad"], out=st["table_grad"])
    if kind == "normfwd":
        return op.forward(st["x"], st["weight"], st["bias"])
    if kind == "normbwd":
        return op.backward(st["grad"], st["x"], st["mean"], st["rstd"], st["weight"], dweight=st["weight_grad"],
                           dbias=st["bias_grad"])
    losses, dlogits = op(st["logits"], st["teacher"], st["index"], temperature=c["temperature"], weights=st["weights"],
                         grad_scale=c["scale"], with_grad=c["grad"])
    return (losses, dlogits) if c["grad"] else (losses,)


def _run_plain(st):
    c = st["case"]
    kind = c["op"]
    if kind == "lookup":
        return (st["weight"][st["ids"]].float() * c["scale"]).to(DTYPES[c["otype"]])
    if kind == "embgrad":
        ids = st["ids"].reshape(-1)
        g = st["grad"].reshape(-1, c["dim"]).float()
        if c["pad"]:
            g = torch.where((ids == 0)[:, None], 0.0, g)
        table = torch.zeros((c["vocab"], c["dim"]), dtype=torch.float32, device=g.device)
        return (table.index_add_(0, ids, g) * c["scale"]).to(DTYPES[c["otype"]])
    if kind == "normfwd":
        x = st["x"].float()
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = torch.rsqrt((d * d).mean(1) + EPS)
        y = d * rstd[:, None] * st["weight"].float() + st["bias"].float()
        return y.to(st["x"].dtype), mean, rstd
    if kind == "normbwd":
        g, w = st["grad"].float(), st["weight"].float()
        xh = (st["x"].float() - st["mean"][:, None]) * st["rstd"][:, None]
        a = g * w
        dx = st["rstd"][:, None] * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
        p = DTYPES[c["ptype"]]
        return dx.to(st["x"].dtype), (g * xh).sum(0).to(p), g.sum(0).to(p)
    t, w = c["temperature"], st["weights"]
    z = st["logits"].float() / t
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    valid = st["index"] >= 0
    at = torch.where(valid, st["index"], 0).long()
    has = valid.any(1) & (w != 0)
    y = torch.where(valid, st["teacher"].float() / t, -math.inf)
    p = torch.exp(y - y.max(1, keepdim=True).values)
    p = p / p.sum(1, keepdim=True)
    logq = z.gather(1, at) - top - torch.log(total)
    part = torch.where(p > 0, p * (torch.log(p) - logq), 0.0)
    losses = torch.where(has, w * (t * t) * part.sum(1), 0.0)
    if not c["grad"]:
        return (losses,)
    q = e / total
    q = q.scatter_add_(1, at, torch.where(valid, -p, 0.0))
    factor = torch.where(has, w * (t * c["scale"]), 0.0)
    return losses, torch.where(has[:, None], q * factor[:, None], 0.0).to(st["logits"].dtype)


# -- the definitions in 64 bits --------------------------------------------------

def exact(case, seed):
    st, c = _inputs(case, seed), case
    op = c["op"]
    if op == "lookup":
        return torch.index_select(st["weight"].double(), 0, st["ids"].reshape(-1).long()).view(
            c["batch"], c["seq"], c["dim"]) * c["scale"]
    if op == "embgrad":
        # the tokens in order, each row of the table the difference of two running sums
        ids = st["ids"].reshape(-1).long()
        g = st["grad"].reshape(-1, c["dim"]).double() * c["scale"]
        if c["pad"]:
            keep = ids != 0
            ids, g = ids[keep], g[keep]
        table = torch.zeros((c["vocab"], c["dim"]), dtype=torch.float64, device="cuda")
        if ids.numel():
            order = torch.argsort(ids, stable=True)
            found, count = torch.unique_consecutive(ids[order], return_counts=True)
            sums = torch.cat([torch.zeros((1, c["dim"]), dtype=torch.float64, device="cuda"), torch.cumsum(g[order], 0)])
            end = torch.cumsum(count, 0)
            table[found] = sums[end] - sums[end - count]
        return table
    if op in ("normfwd", "normbwd"):
        x = st["x"].double()
        w, d = st["weight"].double(), c["dim"]
        if op == "normfwd":
            mean = x.sum(1) / d
            var = ((x - mean[:, None]) ** 2).sum(1) / d
            rstd = 1.0 / torch.sqrt(var + EPS)
            return torch.addcmul(st["bias"].double(), (x - mean[:, None]) * rstd[:, None], w), mean, rstd
        g, mean, rstd = st["grad"].double(), st["mean"].double(), st["rstd"].double()
        xh = (x - mean[:, None]) * rstd[:, None]
        del x
        dw, db = torch.einsum("ij,ij->j", g, xh), g.sum(0)
        g *= w
        s0, s1 = g.sum(1) / d, torch.einsum("ij,ij->i", g, xh) / d
        return (g - s0[:, None] - xh * s1[:, None]) * rstd[:, None], dw, db
    t, n = c["temperature"], c["rows"]
    losses = torch.zeros(n, dtype=torch.float64, device="cuda")
    dz = torch.zeros((n, c["vocab"]), dtype=torch.float64, device="cuda") if c["grad"] else None
    for lo in range(0, n, 512):  # rows are independent: some at a time
        hi = min(n, lo + 512)
        logq = torch.log_softmax(st["logits"][lo:hi].double() / t, 1)
        valid = st["index"][lo:hi] >= 0
        w = st["weights"][lo:hi].double()
        live = valid.any(1) & (w != 0)
        logp = torch.log_softmax(torch.where(valid, st["teacher"][lo:hi].double() / t, -math.inf), 1)
        p = torch.exp(logp)
        at = st["index"][lo:hi].long().clamp(min=0)
        part = torch.where(valid, p * (torch.where(valid, logp, 0.0) - torch.gather(logq, 1, at)), 0.0)
        losses[lo:hi] = torch.where(live, w * t * t * part.sum(1), 0.0)
        if dz is not None:
            target = torch.zeros_like(logq).scatter_add_(1, at, torch.where(valid, p, 0.0))
            dz[lo:hi] = torch.where(live[:, None], (c["scale"] * t) * w[:, None] * (torch.exp(logq) - target), 0.0)
    return (losses, dz) if c["grad"] else (losses,)


# -- what a pass cannot do without -------------------------------------------------

def _distinct(vocab, tokens):
    """How many different rows `tokens` draws of the Zipf law above touch, on average."""
    r = np.arange(1.0, vocab + 1.0)
    p = np.log1p(1.0 / r) / math.log(vocab + 1.0)
    return float(np.sum(-np.expm1(tokens * np.log1p(-p)))) if vocab > 1 else 1.0


def work(case):
    c, op = case, case["op"]
    if op in ("lookup", "embgrad"):
        n, v, d = c["batch"] * c["seq"], c["vocab"], c["dim"]
        ids = n * (4 if c["idtype"] == "i32" else 8)
        if op == "lookup":
            # each row that some token names read once, each output written once
            return {"bytes": ids + _distinct(v, n) * d * SIZE[c["wtype"]] + n * d * SIZE[c["otype"]], "flops": n * d}
        # the gradients of the tokens that are not padding (three quarters of a padded batch), the whole table written once
        live = 0.75 * n if c["pad"] and c["ids"] == "text" else n
        return {"bytes": ids + live * d * SIZE[c["gtype"]] + v * d * SIZE[c["otype"]], "flops": 2 * live * d}
    if op in ("normfwd", "normbwd"):
        n, d, b, p = c["rows"], c["dim"], SIZE[c["xtype"]], SIZE[c["ptype"]]
        if op == "normfwd":
            return {"bytes": 2 * n * d * b + 8 * n + 2 * d * p, "flops": 8 * n * d}
        return {"bytes": 3 * n * d * b + 8 * n + 3 * d * p, "flops": 14 * n * d}
    # logits read once where the row counts, the gradient written once; an exponential counts as one operation
    n, v, live = c["rows"], c["vocab"], c["rows"] * (1.0 - c["masked"])
    entry = SIZE[c["ttype"]] + (4 if c["idtype"] == "i32" else 8)
    grad = n * v * SIZE[c["ztype"]] if c["grad"] else 0
    return {"bytes": live * v * SIZE[c["ztype"]] + grad + n * c["k"] * entry + 8 * n,
            "flops": live * v * (9 if c["grad"] else 5)}
