"""The operators at the two ends of a model measured, where it meets its
vocabulary.

  lookup       rows of the embedding table for a batch of tokens, scaled
  lookup_bwd   the table's gradient: rows of equal tokens summed
  loss         softmax cross entropy of hidden states against a vocabulary,
               from the output projection's weights, without keeping logits
  loss_bwd     its gradients of the hidden states and of the weights, in
               pieces of the vocabulary

Tables, weights and hidden states are BF16, or E4M3 codes under one scale per
tensor.  A token or target outside the vocabulary is padding: its row is
zero, has no loss and adds nothing.

With `own` false, run() computes them from elementary torch operations in 32
bits; with `own` true through the package's entry points.  Both get what
prepare() made from the seed.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
F8 = torch.float8_e4m3fn
PADDING = -100

_LARGEST_FLOPS = 6 * 8192 * 32000 * 4096


def listed():
    return [
        # one decoded token's row of the table: latency alone
        dict(name="lookup, one token", op="lookup", tokens=1, vocab=32000, cols=4096, kind="bf16", scaled=False,
             padding=0),
        # a packed batch that ends in padding, the table kept in 8 bits
        dict(name="lookup, 8-bit table", op="lookup", tokens=8191, vocab=32000, cols=4096, kind="fp8", scaled=True,
             padding=61),
        # the table's gradient in training, for an optimizer that reads BF16
        dict(name="lookup gradient", op="lookup_bwd", tokens=8192, vocab=32000, cols=4096, out="bf16", scaled=True,
             padding=0),
        # an odd batch, an odd vocabulary, the gradient in 32 bits (more is to be added to it)
        dict(name="lookup gradient, odd", op="lookup_bwd", tokens=4099, vocab=50001, cols=2048, out="fp32",
             scaled=False, padding=300),
        # the likelihood of one token
        dict(name="loss, one token", op="loss", rows=1, vocab=32000, cols=4096, kind="bf16", masked=0.0, z=0.0),
        # training
        dict(name="loss, training", op="loss", rows=8192, vocab=32000, cols=4096, kind="bf16", masked=0.0, z=0.0),
        # training with an 8-bit output projection behind a norm that writes E4M3
        dict(name="loss, 8-bit", op="loss", rows=8192, vocab=32000, cols=4096, kind="fp8", masked=0.0, z=0.0),
        # fine-tuning on answers: prompts have no loss; an odd vocabulary, and a penalty on the partition function
        dict(name="loss, masked, odd", op="loss", rows=1021, vocab=50001, cols=2048, kind="bf16", masked=0.4, z=1e-4),
        # a short sequence through a small model
        dict(name="loss gradient, few rows", op="loss_bwd", rows=61, vocab=32000, cols=1024, kind="bf16", masked=0.0,
             z=0.0, piece=32000),
        # fine-tuning on answers
        dict(name="loss gradient, masked, odd", op="loss_bwd", rows=2047, vocab=50001, cols=2048, kind="bf16",
             masked=0.4, z=1e-4, piece=16384),
        # training with an 8-bit output projection
        dict(name="loss gradient, 8-bit", op="loss_bwd", rows=4096, vocab=32000, cols=4096, kind="fp8", masked=0.0,
             z=0.0, piece=8192),
        # training
        dict(name="loss gradient, largest", op="loss_bwd", rows=8192, vocab=32000, cols=4096, kind="bf16", masked=0.0,
             z=0.0, piece=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("lookup", "lookup_bwd", "loss", "loss", "loss_bwd", "loss_bwd"))
    if op in ("lookup", "lookup_bwd"):
        cols = 16 * _log(rng, 8, 512)
        vocab = min(_log(rng, 300, 262144), (1 << 28) // cols)
        tokens = min(_log(rng, 1, 32768), (1 << 26) // cols)
        c = dict(op=op, tokens=tokens, vocab=vocab, cols=cols, scaled=rng.random() < 0.5,
                 padding=rng.choice((0, 0, tokens // 9)))
        if op == "lookup":
            c["kind"] = rng.choice(("bf16", "fp8"))
        else:
            c["out"] = rng.choice(("bf16", "fp32"))
        return c
    kind = rng.choice(("bf16", "bf16", "fp8"))
    unit = 64 if kind == "bf16" else 128
    cols = unit * max(1, _log(rng, 192, 8192) // unit)
    vocab = min(_log(rng, 300, 131072), (1 << 28) // cols)
    rows = max(1, min(_log(rng, 1, 16384), _LARGEST_FLOPS // (6 * vocab * cols), (8192 * 32000) // vocab))
    c = dict(op=op, rows=rows, vocab=vocab, cols=cols, kind=kind, masked=rng.choice((0.0, 0.0, 0.3, 0.6)),
             z=rng.choice((0.0, 1e-4)))
    if op == "loss_bwd":
        c["piece"] = rng.choice((4096, 8192, 16384))
    return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _empty(*shape, dtype):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _tokens(gen, count, vocab):
    """Tokens as text has them: the frequency of the n-th most common one goes with 1/n; the common ones lie scattered."""
    u = torch.rand(count, device="cuda", generator=gen, dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1.0)).long() - 1).clamp(0, vocab - 1)
    stride = next(s for s in (7919, 6997, 5003, 1) if math.gcd(s, vocab) == 1)
    return rank * stride % vocab


def _codes(v):
    """E4M3 codes of FP32 values, saturating."""
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(F8).view(torch.uint8)


def _sequence(c):
    """Rows of a sequence, and how many of them, the first ones, are a prompt without targets."""
    length = min(300, c["rows"])
    return length, int(length * c["masked"])


def prepare(case, seed):
    gen, c, op = _gen(seed), case, case["op"]
    s = dict(c)
    vocab, cols = c["vocab"], c["cols"]
    if op in ("lookup", "lookup_bwd"):
        n = c["tokens"]
        s["ids"] = _tokens(gen, n, vocab)
        if c["padding"]:
            s["ids"][n - c["padding"]:] = PADDING
        s["scale"] = math.sqrt(cols) if c["scaled"] else 1.0
        if op == "lookup":
            table = 0.02 * _normal(gen, vocab, cols)
            s["table_scale"] = 2.0 ** -12 if c["kind"] == "fp8" else 1.0
            s["table"] = _codes(table / s["table_scale"]) if c["kind"] == "fp8" else table.to(torch.bfloat16)
            s["out_rows"] = _empty(n, cols, dtype=torch.bfloat16)
        else:
            s["dy"] = (1e-3 * _normal(gen, n, cols)).to(torch.bfloat16)
            s["dw"] = _empty(vocab, cols, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)
            s["workspace"] = _empty(2 * n * cols + 64 * (n + vocab) + (1 << 22), dtype=torch.uint8)
        return s
    rows, fp8 = c["rows"], c["kind"] == "fp8"
    weight = 0.02 * _normal(gen, vocab, cols)
    targets = _tokens(gen, rows, vocab)
    # hidden states behind a norm, leaning towards their target's row as a model that has learnt something makes them
    x = _normal(gen, rows, cols)
    x += (8.0 / (0.02 * cols)) * torch.rand(rows, 1, device="cuda", generator=gen) * (weight[targets] / 0.02)
    length, prompt = _sequence(c)
    targets[torch.arange(rows, device="cuda") % length < prompt] = PADDING
    s["x_scale"], s["w_scale"] = (2.0 ** -5, 2.0 ** -12) if fp8 else (1.0, 1.0)
    s["x"] = _codes(x / s["x_scale"]) if fp8 else x.to(torch.bfloat16)
    s["w"] = _codes(weight / s["w_scale"]) if fp8 else weight.to(torch.bfloat16)
    s["targets"] = targets
    del x, weight
    if op == "loss":
        s["loss"], s["lse"] = _empty(rows, dtype=torch.float32), _empty(rows, dtype=torch.float32)
        s["workspace"] = _empty(16 * (rows + 256) * (vocab // 64 + 4) + (1 << 22), dtype=torch.uint8)
    else:
        s["lse"] = _plain_loss(s)["lse"]
        # the mean over the rows that have a target
        live = _live(s)
        s["d_loss"] = live.float() / live.sum().clamp(min=1)
        s["dx"] = _empty(rows, cols, dtype=torch.bfloat16)
        s["dw"] = _empty(vocab, cols, dtype=torch.bfloat16)
        piece = min(c["piece"], vocab)
        size = 2 * (rows + 256) * (piece + 256) + 8 * (rows + 256) * cols + 4 * piece * cols + (1 << 26)
        s["workspace"] = _empty(size, dtype=torch.uint8)
    return s


# ------------------------------------------------------------ plain forms

def _values(v, scale):
    return v.view(F8).float() * scale if v.dtype == torch.uint8 else v.float()


def _plain_lookup(s):
    ids = s["ids"]
    live = (ids >= 0) & (ids < s["vocab"])
    rows = _values(s["table"][ids.clamp(0, s["vocab"] - 1)], s["table_scale"]) * s["scale"]
    return torch.where(live[:, None], rows, torch.zeros_like(rows)).to(torch.bfloat16)


def _plain_lookup_bwd(s):
    ids = s["ids"]
    live = (ids >= 0) & (ids < s["vocab"])
    dy = s["dy"].float() * s["scale"]
    dy = torch.where(live[:, None], dy, torch.zeros_like(dy))
    dw = torch.zeros(s["vocab"], s["cols"], device="cuda")
    dw.index_add_(0, ids.clamp(0, s["vocab"] - 1), dy)
    return dw.to(s["dw"].dtype)


def _live(s):
    return (s["targets"] >= 0) & (s["targets"] < s["vocab"])


def _plain_loss(s):
    logits = _values(s["x"], s["x_scale"]) @ _values(s["w"], s["w_scale"]).t()
    top = logits.amax(1, keepdim=True)
    at = logits.gather(1, s["targets"].clamp(0, s["vocab"] - 1)[:, None])[:, 0]
    lse = top[:, 0] + (logits - top).exp_().sum(1).log()
    loss = lse - at + s["z"] * lse * lse
    zero = torch.zeros((), device="cuda")
    return {"loss": torch.where(_live(s), loss, zero), "lse": torch.where(_live(s), lse, zero)}


def _plain_loss_bwd(s):
    x, w = _values(s["x"], s["x_scale"]), _values(s["w"], s["w_scale"])
    live, lse = _live(s)[:, None], s["lse"][:, None]
    d = s["d_loss"][:, None]
    g = (x @ w.t() - lse).exp_() * (d * (1.0 + 2.0 * s["z"] * lse))
    g.scatter_add_(1, s["targets"].clamp(0, s["vocab"] - 1)[:, None], -d)
    g = torch.where(live, g, torch.zeros((), device="cuda"))
    return {"dx": (g @ w).to(torch.bfloat16), "dw": (g.t() @ x).to(torch.bfloat16)}


_PLAIN = {"lookup": _plain_lookup, "lookup_bwd": _plain_lookup_bwd, "loss": _plain_loss, "loss_bwd": _plain_loss_bwd}


# ------------------------------------------------- the package's own calls

_coat = None


def _package():
    global _coat
    if _coat is None:
        from adamw_coat_fp8_amd import coat
        _coat = coat
    return _coat


def _own_lookup(s):
    _package().embedding(s["table"], s["ids"], s["out_rows"], table_scale=s["table_scale"], scale=s["scale"])
    return s["out_rows"]


def _own_lookup_bwd(s):
    _package().embedding_bwd(s["dy"], s["ids"], s["dw"], scale=s["scale"], workspace=s["workspace"])
    return s["dw"]


def _own_loss(s):
    _package().cross_entropy(s["x"], s["w"], s["targets"], s["loss"], s["lse"], x_scale=s["x_scale"],
                             weight_scale=s["w_scale"], z_loss=s["z"], workspace=s["workspace"])
    return {"loss": s["loss"], "lse": s["lse"]}


def _own_loss_bwd(s):
    _package().cross_entropy_bwd(s["d_loss"], s["x"], s["w"], s["targets"], s["lse"], s["dx"], s["dw"],
                                 x_scale=s["x_scale"], weight_scale=s["w_scale"], z_loss=s["z"],
                                 workspace=s["workspace"])
    return {"dx": s["dx"], "dw": s["dw"]}


_OWN = {"lookup": _own_lookup, "lookup_bwd": _own_lookup_bwd, "loss": _own_loss, "loss_bwd": _own_loss_bwd}


def run(state):
    if own:
        return _OWN[state["op"]](state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------- work

def _distinct(count, vocab):
    """How many different tokens _tokens() is expected to give."""
    step = max(1, vocab // 4096)   # (tokens of near frequency together)
    total = 0.0
    for first in range(0, vocab, step):
        n = min(step, vocab - first)
        p = math.log((first + n + 1.0) / (first + 1.0)) / math.log(vocab + 1.0) / n
        total += n * -math.expm1(count * math.log1p(-min(p, 0.999999)))
    return total


def work(case):
    c, op = case, case["op"]
    vocab, cols = c["vocab"], c["cols"]
    if op in ("lookup", "lookup_bwd"):
        n, live = c["tokens"], c["tokens"] - c["padding"]
        if op == "lookup":
            each = 2 if c["kind"] == "bf16" else 1
            return {"bytes": 8 * n + each * cols * _distinct(live, vocab) + 2 * n * cols, "flops": live * cols}
        return {"bytes": 8 * n + 2 * live * cols + (2 if c["out"] == "bf16" else 4) * vocab * cols,
                "flops": live * cols}
    rows, each = c["rows"], 2 if c["kind"] == "bf16" else 1
    length, prompt = _sequence(c)
    live = sum(1 for r in range(rows) if r % length >= prompt)
    product = 2 * live * vocab * cols
    if op == "loss":
        return {"bytes": each * (live + vocab) * cols + 16 * rows, "flops": product}
    return {"bytes": each * (live + vocab) * cols + 2 * (rows + vocab) * cols + 16 * rows, "flops": 3 * product}


# ----------------------------------------------- the definitions in 64 bits

def _table_64():
    """The value of each of the 256 codes (the two NaN codes as 0)."""
    code = torch.arange(256, device="cuda")
    e, m = (code >> 3) & 15, (code & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2(e.double() - 10.0))
    v[[127, 255]] = 0.0
    return torch.where(code >= 128, -v, v)


def _wide(v, scale):
    if v.dtype == torch.uint8:
        return _table_64()[v.long()] * scale
    return v.double()


def exact(case, seed):
    s = prepare(case, seed)
    op, vocab = case["op"], case["vocab"]
    if op in ("lookup", "lookup_bwd"):
        ids = s["ids"]
        keep = [bool(0 <= t < vocab) for t in ids.tolist()]
        keep = torch.tensor(keep, device="cuda")
        if op == "lookup":
            out = torch.zeros(len(ids), case["cols"], dtype=torch.float64, device="cuda")
            out[keep] = _wide(s["table"][ids[keep]], s["table_scale"]) * s["scale"]
            return out
        dw = torch.zeros(vocab, case["cols"], dtype=torch.float64, device="cuda")
        return dw.index_put_((ids[keep],), s["dy"][keep].double() * s["scale"], accumulate=True)
    rows, targets = case["rows"], s["targets"]
    keep = torch.nonzero((targets >= 0) & (targets < vocab))[:, 0]
    x, t = _wide(s["x"][keep], s["x_scale"]), targets[keep]
    step = max(1, min(vocab, (1 << 28) // max(1, len(keep))))
    pieces = [slice(v, min(v + step, vocab)) for v in range(0, vocab, step)]

    def logits(p):
        return x @ _wide(s["w"][p], s["w_scale"]).t()

    if op == "loss":
        lse = torch.full((len(keep),), -math.inf, dtype=torch.float64, device="cuda")
        for p in pieces:
            lse = torch.logaddexp(lse, torch.logsumexp(logits(p), 1)) if len(keep) else lse
        mine = (x * _wide(s["w"][t], s["w_scale"])).sum(1)
        out = {k: torch.zeros(rows, dtype=torch.float64, device="cuda") for k in ("loss", "lse")}
        out["loss"][keep] = lse - mine + case["z"] * lse ** 2
        out["lse"][keep] = lse
        return out
    lse, d = s["lse"].double()[keep], s["d_loss"].double()[keep]
    dx = torch.zeros(rows, case["cols"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(vocab, case["cols"], dtype=torch.float64, device="cuda")
    for p in pieces:
        share = torch.softmax(torch.cat((logits(p), lse[:, None]), 1), 1)   # relative to lse: share / last
        g = share[:, :-1] / share[:, -1:] * (1.0 + 2.0 * case["z"] * lse)[:, None]
        here = torch.nonzero((t >= p.start) & (t < p.stop))[:, 0]
        g[here, t[here] - p.start] -= 1.0
        g *= d[:, None]
        dx[keep] += g @ _wide(s["w"][p], s["w_scale"])
        dw[p] = g.t().contiguous() @ x
    return {"dx": dx, "dw": dw}
