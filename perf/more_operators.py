"""The output layer's losses of a training step, as measured cases.

Two passes over one output layer, logits = hidden @ weight^T, whose gradients
are what the ranks of a data-parallel step then reduce, clip and apply:

  ce       softmax cross entropy against one target a token
  distill  Kullback-Leibler divergence from a teacher's top logits: the teacher's
           distribution is the softmax of a token's k kept logits, the student's
           the softmax of all its logits, both at one temperature; times its square

each with `grads` (gradients of hidden and weight, as in training) or without (as
in evaluation).  Nothing of tokens x vocab is an output.

`keep`: the share of tokens that count; the others have the target -100, or no
teacher entry (ids of -1).  `top`: k.  Teacher lists end early (id -1) in a part of
the rows, as lists cut by probability do.

The record is four floats: loss, tokens counted, nonfinite, factor.  The loss is
the sum of the tokens' losses times the factor, scale / tokens counted ("mean")
or scale ("sum"); the gradients are the loss's.
"""

import math

import torch

own = False

IGNORE = -100


def _case(name, op, tokens, hidden, vocab, dtype, **more):
    c = {"name": name, "op": op, "tokens": tokens, "hidden": hidden, "vocab": vocab, "dtype": dtype, "grads": True,
         "keep": 1.0, "reduction": "mean", "scale": 1.0, "top": 0, "temperature": 1.0}
    c.update(more)
    return c


def listed():
    return [
        # one token of a small model scored: launches and one dependent chain
        _case("ce-one-token", "ce", 1, 640, 10007, "bfloat16", grads=False),
        # a toy model's training step of odd sizes: latency, rows off every vector alignment
        _case("ce-toy-odd", "ce", 37, 129, 2003, "float32"),
        # a small float32 model
        _case("ce-fp32", "ce", 515, 515, 10007, "float32", reduction="sum", scale=1.0 / 515),
        # perplexity over a long document
        _case("ce-eval-16k", "ce", 16384, 1024, 32003, "bfloat16", grads=False),
        # fine-tuning on answers: half of the tokens are prompt or padding; odd sizes
        _case("ce-half-masked", "ce", 8191, 1023, 32003, "bfloat16", keep=0.5),
        # an ordinary micro-batch
        _case("ce-train-4k", "ce", 4096, 2048, 50001, "bfloat16"),
        # a large micro-batch under a large vocabulary, its loss scaled
        _case("ce-train-8k-large", "ce", 8192, 4096, 128000, "bfloat16", scale=1024.0),
        # a few tokens' update of a small student: latency
        _case("distill-few", "distill", 5, 192, 4001, "bfloat16", top=8),
        # a float32 student, softened
        _case("distill-fp32", "distill", 300, 256, 5003, "float32", top=16, temperature=2.0),
        # odd sizes, a third of the tokens without a teacher
        _case("distill-odd-masked", "distill", 3001, 771, 10007, "bfloat16", top=33, temperature=2.0, keep=0.67),
        # an ordinary micro-batch with 64 kept logits
        _case("distill-2k", "distill", 2048, 2048, 50001, "bfloat16", top=64),
        # a large one
        _case("distill-4k-large", "distill", 4096, 4096, 65537, "bfloat16", top=128, reduction="sum", scale=1.0 / 4096),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ce", "distill"])
    while True:
        dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
        tokens, hidden, vocab = _spread(rng, 1, 16384), _spread(rng, 64, 4096), _spread(rng, 500, 128000)
        if rng.random() < 0.5:
            hidden = max(64, hidden // 64 * 64)
        c = {"op": op, "tokens": tokens, "hidden": hidden, "vocab": vocab, "dtype": dtype,
             "grads": rng.random() < 0.75, "keep": rng.choice([1.0, 1.0, 0.9, 0.4]),
             "reduction": rng.choice(["mean", "sum"]), "scale": rng.choice([1.0, 0.25, 1.0 / 300, 1024.0]),
             "top": _spread(rng, 1, 128) if op == "distill" else 0,
             "temperature": rng.choice([1.0, 1.0, 2.0, 4.0]) if op == "distill" else 1.0}
        most = max(work(x)["flops"] for x in listed() if x["op"] == op and x["dtype"] == dtype)
        if work(c)["flops"] <= most:
            return c


# ---------------------------------------------------------------- inputs

def _dtype(name):
    return getattr(torch, name)


def _inputs(case, seed):
    """Hidden states, weights and targets (or a teacher's lists), from the seed
    alone.  A token's hidden state leans towards what it should predict, by an
    amount of its own: a trained model is sure of some tokens and not of others."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, d, v, k = case["tokens"], case["hidden"], case["vocab"], case["top"]
    weight = torch.randn(v, d, generator=g, device="cuda").mul_(1.25 / math.sqrt(d)).to(_dtype(case["dtype"]))
    hidden = torch.randn(n, d, generator=g, device="cuda")
    s = {"case": case, "weight": weight}
    counts = torch.rand(n, generator=g, device="cuda") < case["keep"]
    if case["op"] == "ce":
        best = torch.randint(v, (n,), generator=g, device="cuda")
        s["targets"] = torch.where(counts, best, IGNORE)
    else:
        step = torch.randint(1, max(2, v // k), (n, 1), generator=g, device="cuda")
        first = torch.randint(v, (n, 1), generator=g, device="cuda")
        ids = (first + step * torch.arange(k, device="cuda")) % v
        best = ids[:, 0]
        drops = -torch.log(1.0 - torch.rand(n, k, generator=g, device="cuda")) * (4.0 / k)
        drops[:, 0] = 0.0
        s["teacher"] = (18.0 - torch.cumsum(drops, 1)).to(_dtype(case["dtype"]))
        length = torch.where(torch.rand(n, generator=g, device="cuda") < 0.3,
                             torch.randint(1, k + 1, (n,), generator=g, device="cuda"), k)
        there = (torch.arange(k, device="cuda") < length[:, None]) & counts[:, None]
        s["ids"] = torch.where(there, ids, -1)
    lean = torch.rand(n, 1, generator=g, device="cuda") * (14.0 / 1.5625)
    hidden += lean * weight[best].float()
    s["hidden"] = hidden.to(_dtype(case["dtype"]))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    n = case["tokens"]
    s["losses"] = torch.zeros(n, device="cuda")
    s["grad_hidden"] = torch.zeros_like(s["hidden"]) if case["grads"] else None
    s["grad_weight"] = torch.zeros_like(s["weight"]) if case["grads"] else None
    if own:
        import collective_reduction_gb300 as ar
        s["loss"] = ar.OutputLoss(n, case["hidden"], case["vocab"], case["dtype"], top=case["top"])
    return s


# ---------------------------------------------------------------- one pass

def _outputs(s, record):
    out = {"record": record, "losses": s["losses"]}
    if s["case"]["grads"]:
        out.update(grad_hidden=s["grad_hidden"], grad_weight=s["grad_weight"])
    return out


def _finish(s, losses, counted, zgrad):
    """The record, and the gradients from those of the logits before the factor."""
    case = s["case"]
    n = counted.sum()
    factor = case["scale"] / n.clamp(min=1).double() if case["reduction"] == "mean" else \
        torch.full((), case["scale"], dtype=torch.float64, device="cuda")
    loss = losses.double().sum() * factor
    s["losses"].copy_(losses)
    if zgrad is not None:
        zgrad *= factor.float()
        s["grad_hidden"].copy_(zgrad @ s["weight"].float())
        s["grad_weight"].copy_(zgrad.t() @ s["hidden"].float())
    bad = 1.0 - torch.isfinite(losses).all().double()
    return torch.stack([loss, n.double(), bad, factor]).float()


def _plain_ce(s):
    targets = s["targets"]
    counted = targets >= 0
    z = s["hidden"].float() @ s["weight"].float().t()
    top = z.amax(1, keepdim=True)
    at = targets.clamp(min=0)[:, None]
    mine = z.gather(1, at) - top
    q = z.sub_(top).exp_()
    total = q.sum(1, keepdim=True)
    losses = torch.where(counted, (total.log() - mine)[:, 0], 0.0)
    if s["case"]["grads"]:
        q /= total
        q.scatter_add_(1, at, torch.full_like(mine, -1.0))
        q *= counted[:, None]
    return _finish(s, losses, counted, q if s["case"]["grads"] else None)


def _plain_distill(s):
    t, ids = s["case"]["temperature"], s["ids"]
    there = ids >= 0
    counted = there.any(1)
    u = torch.where(there, s["teacher"].float() / t, -math.inf)
    u = torch.where(there, u - torch.where(counted, u.amax(1), 0.0)[:, None], -math.inf)
    p = u.exp()
    mass = p.sum(1, keepdim=True).clamp(min=1e-30)
    p = p / mass
    logp = u - mass.log()
    z = s["hidden"].float() @ s["weight"].float().t()
    z /= t
    top = z.amax(1, keepdim=True)
    at = ids.clamp(min=0)
    mine = z.gather(1, at) - top
    q = z.sub_(top).exp_()
    total = q.sum(1, keepdim=True)
    terms = torch.where(there, p * (logp - (mine - total.log())), 0.0)
    losses = terms.sum(1) * (t * t)
    if s["case"]["grads"]:
        q /= total
        q.scatter_add_(1, at, -p)
        q *= counted[:, None] * t
    return _finish(s, losses, counted, q if s["case"]["grads"] else None)


def run(s):
    case = s["case"]
    if own:
        more = {"reduction": case["reduction"], "scale": case["scale"], "losses": s["losses"],
                "grad_hidden": s["grad_hidden"], "grad_weight": s["grad_weight"]}
        if case["op"] == "ce":
            return _outputs(s, s["loss"].cross_entropy(s["hidden"], s["weight"], s["targets"], ignore_index=IGNORE, **more))
        return _outputs(s, s["loss"].distill(s["hidden"], s["weight"], s["ids"], s["teacher"],
                                             temperature=case["temperature"], **more))
    return _outputs(s, _plain_ce(s) if case["op"] == "ce" else _plain_distill(s))


def work(case):
    n, d, v, k = case["tokens"], case["hidden"], case["vocab"], case["top"]
    es = 2 if case["dtype"] == "bfloat16" else 4
    counted = max(1, int(round(n * case["keep"])))  # the others' hidden states need not be read
    lists = n * 8 if case["op"] == "ce" else n * k * (8 + es)
    read = es * (counted * d + v * d) + lists
    if not case["grads"]:
        return {"bytes": read + 4 * n, "flops": 2 * counted * v * d}
    return {"bytes": read + es * (n * d + v * d) + 4 * n, "flops": 6 * counted * v * d}


# ---------------------------------------------------------------- the definition in 64 bits

EXACT_FLOPS = 6e12  # float64 products run at about 1 TFLOP/s


def exact(case, seed):
    n, v = case["tokens"], case["vocab"]
    if (6 if case["grads"] else 2) * n * v * case["hidden"] > EXACT_FLOPS:
        return None
    s = _inputs(case, seed)
    x, w = s["hidden"].to(torch.float64), s["weight"].to(torch.float64)
    t = float(case["temperature"])
    if case["op"] == "ce":
        ids, share = s["targets"][:, None], (s["targets"] >= 0).to(torch.float64)[:, None]
    else:
        ids = s["ids"]
        share = torch.softmax(torch.where(ids >= 0, s["teacher"].to(torch.float64) / t, -1e300), 1) * (ids >= 0)
    counted = [i for i, c in enumerate((ids >= 0).any(1).tolist()) if c]
    factor = case["scale"] / max(1, len(counted)) if case["reduction"] == "mean" else case["scale"]
    losses = torch.zeros(n, dtype=torch.float64, device="cuda")
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    step = max(1, (1 << 28) // v)
    for a in range(0, len(counted), step):  # rows at a time: tokens x vocab in 64 bits is large
        rows = torch.tensor(counted[a:a + step], device="cuda")
        target = torch.zeros(len(rows), v, dtype=torch.float64, device="cuda")
        target.scatter_add_(1, ids[rows].clamp(min=0), share[rows])
        logq = torch.log_softmax(x[rows] @ w.t() / t, 1)
        losses[rows] = t * t * (torch.xlogy(target, target) - target * logq).sum(1)
        if case["grads"]:
            dz = logq.exp_().sub_(target).mul_(t * factor)
            dx[rows] = dz @ w
            dw += dz.t() @ x[rows]
    out = {"record": torch.tensor([math.fsum(losses.tolist()) * factor, len(counted), 0.0, factor], dtype=torch.float64),
           "losses": losses}
    if case["grads"]:
        out.update(grad_hidden=dx, grad_weight=dw)
    return out
