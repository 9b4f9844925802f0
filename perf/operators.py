"""What follows the gradients' allreduce in a training step, as measured cases.

Four passes over the tensors of one training program:

  norm   the global gradient norm over many tensors, with its record
  clip   the norm, then every gradient scaled by the record's factor
  adamw  one AdamW update of parameters and moments
  step   the norm's record, then AdamW reading its clip factor on the device

A case describes the tensors as a stack of equal layers: an embedding of
`vocab` x `hidden`, and per layer four hidden x hidden matrices, two
hidden x ffn matrices and four vectors of `hidden`, then a last vector.  They
are views of one flat buffer per element type, as in a bucketed gradient
buffer: `align` is the element multiple every view starts at (1: packed tight,
so odd sizes leave most views off any vector alignment).
`grad`: the gradients' element type; "mixed" keeps matrices in bfloat16 and
vectors in float32.  `param`: the parameters'; moments are always float32.

The record is four floats: norm, scale, nonfinite, clipped.  With the
pre-scale c (one over the loss scale or the rank count), norm = c ||g||,
clipped = norm > max_norm, scale = c max_norm / norm if clipped else c.

Clipping is measured into other tensors (`out`): in place, the second pass
over one state would find its gradients clipped already and do less.
"""

import math

import torch

own = False

NORM_VECTORS = 4  # vectors of `hidden` in a layer: two norms' scales, two biases
BETA1, BETA2, EPS, LR, DECAY, STEP = 0.9, 0.95, 1e-8, 3e-4, 0.1, 1000


def _case(name, op, layers, hidden, ffn, vocab, grad, **more):
    c = {"name": name, "op": op, "layers": layers, "hidden": hidden, "ffn": ffn, "vocab": vocab, "matrices": True,
         "grad": grad, "align": 64, "kind": "l2", "pre_scale": 1.0, "max_norm": 1.0, "per_tensor": False}
    c.update(more)
    return c


def listed():
    return [
        # the vectors alone of a small model: what a parameter group without decay holds; latency
        _case("norm-vectors", "norm", 4, 515, 0, 0, "float32", matrices=False),
        # one gradient bucket of about 25 MB, the usual size of a data-parallel bucket
        _case("norm-bucket-25mb", "norm", 1, 640, 2560, 2003, "float32"),
        # a bf16 gradient buffer of odd sizes packed tight, with the norm of every tensor for the log
        _case("norm-bf16-packed", "norm", 24, 1023, 4093, 32003, "bfloat16", align=1, per_tensor=True),
        # the whole gradient of a model of two billion parameters, bf16 with its vectors in fp32
        _case("norm-mixed-2g", "norm", 10, 4096, 16384, 32000, "mixed"),
        # a toy model's gradient: launches and one dependent chain
        _case("clip-toy", "clip", 1, 96, 384, 0, "float32", out="float32"),
        # a gradient that still fits the L2 cache between the norm and the scaling
        _case("clip-96mb", "clip", 2, 1000, 4000, 0, "float32", out="float32", align=1),
        # bf16 model gradients unscaled and clipped into the fp32 gradients an optimizer keeps
        _case("clip-bf16-to-fp32", "clip", 24, 1024, 4096, 50001, "bfloat16", out="float32", pre_scale=1.0 / 1024),
        # a large fp32 gradient
        _case("clip-670m", "clip", 12, 2048, 8192, 32000, "float32", out="float32"),
        # a small model's update
        _case("adamw-small", "adamw", 2, 129, 515, 0, "float32", param="float32", copies=False),
        # mixed precision: bf16 gradients, fp32 master parameters, bf16 copies for the forward
        _case("adamw-bf16-copies", "adamw", 12, 1024, 4096, 32003, "bfloat16", param="float32", copies=True),
        # norm, then the update: bf16 parameters and gradients of odd sizes packed tight
        _case("step-bf16-packed", "step", 16, 771, 3083, 10007, "bfloat16", param="bfloat16", copies=False, align=1),
        # norm, then the update, of a billion fp32 parameters
        _case("step-fp32-1g", "step", 18, 2048, 8192, 50001, "float32", param="float32", copies=False),
    ]


def draw(rng):
    while True:
        op = rng.choice(["norm", "clip", "adamw", "step"])
        most = max(work(c)["bytes"] for c in listed() if c["op"] == op)
        grad = rng.choice(["float32", "bfloat16", "mixed"])
        hidden = int(round(math.exp(rng.uniform(math.log(48), math.log(4096)))))
        if rng.random() < 0.5:
            hidden = max(64, hidden // 64 * 64)
        ffn = hidden * rng.choice([2, 4]) + rng.choice([0, 0, 1, 3])
        layers = int(round(math.exp(rng.uniform(0.0, math.log(40)))))
        vocab = rng.choice([0, int(round(math.exp(rng.uniform(math.log(500), math.log(60000)))))])
        more = {"align": rng.choice([1, 1, 4, 64]), "kind": rng.choice(["l2", "l2", "max"]),
                "pre_scale": rng.choice([1.0, 0.125, 1.0 / 3, 1.0 / 1024]),
                "max_norm": rng.choice([1.0, 0.25]), "per_tensor": op in ("norm", "clip") and rng.random() < 0.3}
        if op == "clip":
            more["out"] = rng.choice(["float32", "same"])
        if op in ("adamw", "step"):
            more["param"] = rng.choice(["float32", "float32", "bfloat16"])
            more["copies"] = more["param"] == "float32" and rng.random() < 0.5
        if op == "norm" and rng.random() < 0.15:
            more["matrices"] = False
        c = _case("", op, layers, hidden, ffn, vocab, grad, **more)
        del c["name"]
        if 3072 not in (hidden, ffn, vocab, 2 * hidden, 4 * hidden) and work(c)["bytes"] <= most:
            return c


# ---------------------------------------------------------------- the tensors of a case

def _shapes(case):
    """[(elements, is_vector)] of every tensor, in the model's order."""
    h, f = case["hidden"], case["ffn"]
    out = [(case["vocab"] * h, False)] if case["vocab"] and case["matrices"] else []
    for _ in range(case["layers"]):
        out += [(h, True)] * NORM_VECTORS
        if case["matrices"]:
            out += [(h * h, False)] * 4 + [(h * f, False)] * 2
    return out + [(h, True)]


def _grad_types(case):
    return [case["grad"] if case["grad"] != "mixed" else "float32" if vec else "bfloat16" for _, vec in _shapes(case)]


def _out_types(case):
    t = _grad_types(case)
    return t if case["out"] == "same" else [case["out"]] * len(t)


_TORCH = {"float32": torch.float32, "bfloat16": torch.bfloat16}
_BYTES = {"float32": 4, "bfloat16": 2}


class _Flat:
    """One flat buffer per element type and the tensors' views of them."""

    def __init__(self, sizes, types, align, dtype=None):
        place, used = [], {}
        for n, t in zip(sizes, types):
            at = -(-used.get(t, 0) // align) * align
            place.append((t, at))
            used[t] = at + n
        self.buffers = {t: torch.zeros(n, dtype=dtype or _TORCH[t], device="cuda") for t, n in used.items()}
        self.views = [self.buffers[t][at:at + n] for (t, at), n in zip(place, sizes)]

    def all(self):
        return [self.buffers[t] for t in sorted(self.buffers)]


def _inputs(case, seed):
    """The flat buffers before the pass, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    shapes = _shapes(case)
    sizes, n = [s for s, _ in shapes], len(shapes)

    def normal(flat, sigma, square=False):
        for t in sorted(flat.buffers):
            b = flat.buffers[t]
            x = b if b.dtype == torch.float32 else torch.empty_like(b, dtype=torch.float32)
            x.normal_(0.0, sigma, generator=g)
            if square:
                x.square_()
            if x is not b:
                b.copy_(x)
        return flat

    total = sum(sizes)
    # a gradient whose scaled norm is about twice the bound of the usual case, its tensors of unlike sizes
    sigma = 2.0 / (case["pre_scale"] * (math.sqrt(total) if case["kind"] == "l2" else 5.0))
    s = {"case": case, "sizes": sizes, "grads": normal(_Flat(sizes, _grad_types(case), case["align"]), sigma)}
    for i, v in enumerate(s["grads"].views):
        if i % 3 == 1 and shapes[i][1]:
            v.mul_(0.25)
    if case["op"] == "clip":
        s["outs"] = _Flat(sizes, _out_types(case), case["align"])
    if case["op"] in ("adamw", "step"):
        s["params"] = normal(_Flat(sizes, [case["param"]] * n, 64), 0.02)
        s["m"] = normal(_Flat(sizes, ["float32"] * n, 64), 0.3 * sigma)
        s["v"] = normal(_Flat(sizes, ["float32"] * n, 64), sigma, square=True)
        s["copies"] = _Flat(sizes, ["bfloat16"] * n, 64) if case["copies"] else None
        s["decay"] = [0.0 if vec else 1.0 for _, vec in shapes]  # vectors do not decay
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import collective_reduction_gb300 as ar
        if case["op"] != "adamw":
            s["plan"] = ar.Grads(s["grads"].views, out=s["outs"].views if case["op"] == "clip" else None)
            if case["per_tensor"]:
                s["norms"] = torch.empty(len(s["sizes"]), device="cuda")
        if case["op"] in ("adamw", "step"):
            s["adamw"] = ar.AdamW(s["params"].views, s["grads"].views, s["m"].views, s["v"].views,
                                  copies=s["copies"].views if s["copies"] else None, decay=s["decay"])
    return s


# ---------------------------------------------------------------- one pass

def _plain_norm(s):
    """The record and the norm of every tensor."""
    case, each = s["case"], []
    for g in s["grads"].views:
        x = g.float()
        each.append((x * x).sum() if case["kind"] == "l2" else x.abs().max())
    each = torch.stack(each)
    c = case["pre_scale"]
    norm = c * (each.sum().sqrt() if case["kind"] == "l2" else each.max())
    norms = c * (each.sqrt() if case["kind"] == "l2" else each)
    nonfinite = ~torch.isfinite(norm)
    clipped = (norm > case["max_norm"]) & ~nonfinite
    scale = torch.where(clipped, c * case["max_norm"] / norm, torch.full_like(norm, c))
    return torch.stack([norm, scale, nonfinite.float(), clipped.float()]), norms


def _plain_adamw(s, scale):
    c1, c2 = 1.0 - BETA1 ** STEP, 1.0 - BETA2 ** STEP
    copies = s["copies"].views if s["copies"] else [None] * len(s["sizes"])
    for p, g, m, v, w, d in zip(s["params"].views, s["grads"].views, s["m"].views, s["v"].views, copies, s["decay"]):
        x = g.float() * scale if scale is not None else g.float()
        m.mul_(BETA1).add_(x * (1.0 - BETA1))
        v.mul_(BETA2).add_(x * x * (1.0 - BETA2))
        q = p.float() * (1.0 - LR * DECAY * d) - (LR / c1) * m / ((v / c2).sqrt() + EPS)
        p.copy_(q)
        if w is not None:
            w.copy_(q)


def _outputs(s, record, norms):
    case, out = s["case"], {}
    if record is not None:
        out["record"] = record
    if case["per_tensor"]:
        out["norms"] = norms
    if case["op"] == "clip":
        out["out"] = s["outs"].all()
    if case["op"] in ("adamw", "step"):
        out.update(params=s["params"].all(), m=s["m"].all(), v=s["v"].all())
        if s["copies"]:
            out["copies"] = s["copies"].all()
    return out


def run(s):
    case, record, norms = s["case"], None, s.get("norms")
    if own:
        how = {"kind": case["kind"], "pre_scale": case["pre_scale"]}
        if case["op"] == "clip":
            record = s["plan"].clip(case["max_norm"], per_tensor=norms, **how)
        elif case["op"] != "adamw":
            record = s["plan"].norm(max_norm=case["max_norm"], per_tensor=norms, **how)
        if case["op"] in ("adamw", "step"):
            s["adamw"].step(STEP, lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY, clip=record)
        return _outputs(s, record, norms)
    if case["op"] != "adamw":
        record, norms = _plain_norm(s)
    if case["op"] == "clip":
        for g, o in zip(s["grads"].views, s["outs"].views):
            o.copy_(g.float() * record[1])
    if case["op"] in ("adamw", "step"):
        _plain_adamw(s, record[1] if record is not None else None)
    return _outputs(s, record, norms)


def work(case):
    shapes = _shapes(case)
    n = sum(k for k, _ in shapes)
    grads = sum(k * _BYTES[t] for (k, _), t in zip(shapes, _grad_types(case)))
    if case["op"] == "norm":
        return {"bytes": grads, "flops": 2 * n}
    if case["op"] == "clip":
        return {"bytes": grads + sum(k * _BYTES[t] for (k, _), t in zip(shapes, _out_types(case))), "flops": 3 * n}
    per = 2 * (_BYTES[case["param"]] + 8) + (2 if case["copies"] else 0)
    return {"bytes": grads + n * per, "flops": (18 if case["op"] == "step" else 15) * n}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    sizes, c, bound = s["sizes"], case["pre_scale"], case["max_norm"]
    out, scale = {}, 1.0
    if case["op"] != "adamw":
        tops, squares = [], []
        for g in s["grads"].views:
            d = g.to(torch.float64)
            tops.append(float(d.abs().amax()))
            squares.append(float(torch.dot(d, d)))
        if case["kind"] == "l2":
            norm, norms = c * math.sqrt(math.fsum(squares)), [c * math.sqrt(q) for q in squares]
        else:
            norm, norms = c * max(tops), [c * t for t in tops]
        clipped = norm > bound
        scale = c * bound / norm if clipped else c
        out["record"] = torch.tensor([norm, scale, 0.0, float(clipped)], dtype=torch.float64)
        if case["per_tensor"]:
            out["norms"] = torch.tensor(norms, dtype=torch.float64)
    if case["op"] == "clip":
        flat = _Flat(sizes, _out_types(case), case["align"], dtype=torch.float64)
        for g, o in zip(s["grads"].views, flat.views):
            torch.mul(g.to(torch.float64), scale, out=o)
        out["out"] = flat.all()
    if case["op"] in ("adamw", "step"):
        types = ["float32"] * len(sizes)
        ptypes = [case["param"]] * len(sizes)
        P, M, V = (_Flat(sizes, t, 64, dtype=torch.float64) for t in (ptypes, types, types))
        for new, old in ((P, s["params"]), (M, s["m"]), (V, s["v"])):
            for t in new.buffers:  # what lies between the tensors stays
                new.buffers[t].copy_(old.buffers[t])
        for i, d in enumerate(s["decay"]):
            g = s["grads"].views[i].to(torch.float64).mul_(scale)
            M.views[i].copy_(s["m"].views[i].to(torch.float64) * BETA1 + g * (1.0 - BETA1))
            V.views[i].copy_(s["v"].views[i].to(torch.float64) * BETA2 + g.square() * (1.0 - BETA2))
            denominator = (V.views[i] / (1.0 - BETA2 ** STEP)).sqrt() + EPS
            update = M.views[i] / (1.0 - BETA1 ** STEP) / denominator
            P.views[i].copy_(s["params"].views[i].to(torch.float64) * (1.0 - LR * DECAY * d) - LR * update)
        out.update(params=P.all(), m=M.all(), v=V.all())
        if case["copies"]:
            W = _Flat(sizes, ["bfloat16"] * len(sizes), 64, dtype=torch.float64)
            for w, p in zip(W.views, P.views):
                w.copy_(p)
            out["copies"] = W.all()
    return out
