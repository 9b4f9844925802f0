"""Gradient norm, clipping and AdamW over many tensors, against their
definitions in 64 bits.

Tolerances, in units of u = 2^-24 (float32's rounding), derived from the
kernels' arithmetic and not from their output:

* L2 norm.  A value's square enters a float32 sum of at most 16 fused
  multiply-adds and 2 more additions; all terms are positive, so the group is
  off by at most 18 u relative, everything after it is float64, the root halves
  it and the result rounds once: 10 u.  The scale is one more rounding: 11 u.
* Max norm: exact but for the product with the pre-scale, rounded once: 1 u
  (the scale, a quotient in float64: 1 u).
* Clipped values: exactly round(scale * g) for the scale in the record.
* AdamW, with M = |b1 m| + |(1 - b1) g| and g = s grad: the constants, g, two
  products and an fma round: m is off by at most 6 u M, v by 8 u v.  The
  denominator (v's half, root, constant, fma) is off by 8 u, the quotient with
  its product and constants by 16 u U, U = lr / bc1 M / denominator; the decay
  term d = lr wd p by 3 u d; the last subtraction and the store round once:
  u |p|, or 2^-8 |p| + u |p| in bfloat16.
"""

import ctypes
import math
import os

import pytest

import collective_reduction_gb300 as ar

U = 2.0 ** -24
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    return ensure_built()


# ------------------------------------------------------------------ host only

@pytest.mark.parametrize("counts", [[], [0], [1], [0, 5, 0, 0, 7], [4095], [4096], [4097], [3 * 4096 + 1, 8192, 2],
                                    [1] * 3000, [(1 << 32) + 5, 3]])
def test_ranges_tile_every_tensor(counts):
    info = ar.tensors_lowering(counts, ["float32"] * len(counts))
    e = info["item_elems"]
    assert info["tiling_ok"] == 1 and info["n_tensors"] == len(counts) and info["elems"] == sum(counts)
    assert info["n_items"] == sum(-(-c // e) for c in counts)


def test_layout_refusals():
    def status(*a):
        with pytest.raises(ar.ArError) as e:
            ar.tensors_lowering(*a)
        return e.value.name
    assert status([4], ["int32"]) == "AR_ERR_UNSUPPORTED"
    assert status([1 << 41], ["float32"]) == "AR_ERR_UNSUPPORTED"
    assert status([1 << 39] * 3, ["bfloat16"] * 3) == "AR_ERR_UNSUPPORTED"
    assert status([1] * ((1 << 20) + 1), ["float32"] * ((1 << 20) + 1)) == "AR_ERR_UNSUPPORTED"
    L, info = ar.lib(), ar.TensorsInfo()
    one, bad = (ctypes.c_uint64 * 1)(4), (ctypes.c_int * 1)(9)
    assert L.ar_tensors_lowering(1, one, bad, ctypes.byref(info)) == 1
    assert L.ar_tensors_lowering(-1, one, bad, ctypes.byref(info)) == 1
    assert L.ar_tensors_lowering(1, None, bad, ctypes.byref(info)) == 1
    assert L.ar_tensors_lowering(1, one, bad, None) == 1


def test_null_handles_are_refused():
    L, info, p, h = ar.lib(), ar.TensorsInfo(), ar.AdamWParams(1, 1e-3, 0.9, 0.99, 1e-8, 0.0), ctypes.c_void_p()
    assert L.ar_grads_query(None, ctypes.byref(info)) == 1
    assert L.ar_grads_destroy(None) == 1
    assert L.ar_adamw_query(None, ctypes.byref(info)) == 1
    assert L.ar_adamw_destroy(None) == 1
    assert L.ar_grad_norm(None, 0, 1.0, 1.0, None, None, None) == 1
    assert L.ar_grad_clip(None, 0, 1.0, 1.0, None, None, None) == 1
    assert L.ar_adamw_step(None, ctypes.byref(p), None, None) == 1
    assert L.ar_adamw_step_counted(None, ctypes.byref(p), None, None, None, None) == 1
    assert L.ar_grads_create(1, None, None, None, None, None, ctypes.byref(h)) == 1
    assert L.ar_grads_create(0, None, None, None, None, None, None) == 1
    assert L.ar_adamw_create(1, None, None, None, None, None, None, None, None, None, ctypes.byref(h)) == 1


def test_binding_refuses_what_it_cannot_bind():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        ar.Grads([torch.zeros(4)])
    with pytest.raises(ValueError, match="element type"):
        ar.Grads([torch.zeros(4, dtype=torch.float16)])
    assert ar._layout(torch.zeros(3, 4)) == "contiguous"
    assert ar._layout(torch.zeros(3, 4).t()) == (1, 4)
    assert ar._layout(torch.zeros(2, 3, 4).permute(2, 0, 1)) == (1, 12, 4)
    assert ar._layout(torch.zeros(3, 8)[:, ::2]) is None
    assert ar._layout(torch.zeros(3, 8)[:, :5]) is None
    assert ar._layout(torch.zeros(1).expand(6)) is None


# --------------------------------------------------------------------- on a GPU

DT = {"float32": 4, "bfloat16": 2}


def tdt(name):
    import torch
    return getattr(torch, name)


class Tensors:
    """Views of guarded device buffers: tensor i of sizes[i] elements lies
    `offset` elements past a 256-byte boundary, sentinels on both sides."""

    def __init__(self, sizes, types, offset=0, seed=0, sigma=1.0, square=False):
        import torch
        g = torch.Generator().manual_seed(seed)
        types = [types] * len(sizes) if isinstance(types, str) else types
        self.views, self.big, self.offset = [], [], offset
        for n, t in zip(sizes, types):
            x = torch.randn(n, generator=g, dtype=torch.float64) * sigma
            big = torch.full((256 + offset + n + 256,), -7.0, dtype=tdt(t), device="cuda")
            v = big[256 + offset:256 + offset + n]
            v.copy_((x * x if square else x).to(tdt(t)))
            self.views.append(v)
            self.big.append(big)

    def wide(self):
        import torch
        return [v.to(torch.float64).cpu() for v in self.views]

    def host(self):
        return [v.cpu().clone() for v in self.views]

    def check_guards(self):
        for b, v in zip(self.big, self.views):
            lead = 256 + self.offset
            assert bool((b[:lead] == -7.0).all()) and bool((b[lead + v.numel():] == -7.0).all())


def true_norms(wide, kind, c):
    import torch
    if kind == "max":
        each = [c * float(x.abs().max()) if x.numel() else 0.0 for x in wide]
        return max(each, default=0.0), each
    each = [float(torch.dot(x, x)) for x in wide]
    return c * math.sqrt(math.fsum(each)), [c * math.sqrt(s) for s in each]


def assert_close(got, want, rel, what):
    assert abs(got - want) <= rel * abs(want) + 2.0 ** -150, (what, got, want)


SIZES = {
    "one": [1],
    "tiny": [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17],
    "empties": [0, 33, 0, 0, 1, 0],
    "warp-edges": [31, 32, 33, 127, 128, 129, 255, 256, 257, 1023, 1024, 1025, 2047, 2049],
    "item-edges": [4095, 4096, 4097, 8191, 8193, 12289],
    "ragged": [100003, 17, 70001, 5, 0, 3001],
    "many": [37] * 400,
    "long": [5000011, 64],
}
TYPES = ["float32", "bfloat16", "mixed"]


def types_of(name, n):
    return [name] * n if name != "mixed" else [("float32", "bfloat16")[i % 2] for i in range(n)]


@gpu
@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("sizes", list(SIZES))
def test_norms(sizes, types, offset):
    import torch
    n = SIZES[sizes]
    t = Tensors(n, types_of(types, len(n)), offset, seed=len(n) + offset)
    wide, before = t.wide(), t.host()
    h = ar.Grads(t.views)
    for kind, c in (("l2", 1.0), ("max", 1.0), ("l2", 1.0 / 3), ("max", 0.125)):
        norm, each = true_norms(wide, kind, c)
        tol = 10 * U if kind == "l2" else U
        per = torch.full((len(n) + 1,), -7.0, device="cuda")
        rec = h.norm(max_norm=0.5 * norm, kind=kind, pre_scale=c, per_tensor=per).tolist()
        assert_close(rec[0], norm, tol, kind)
        assert_close(rec[1], 0.5 * c, tol + U, "scale")
        assert rec[2:] == [0.0, 1.0 if norm > 0 else 0.0]
        for i, (got, want) in enumerate(zip(per.tolist(), each)):
            assert_close(got, want, tol, (kind, i))
        assert per[len(n)].item() == -7.0
        rec = h.norm(max_norm=2.0 * norm + 1.0, kind=kind, pre_scale=c, result=torch.empty(4, device="cuda")).tolist()
        assert_close(rec[1], c, U, "unclipped scale")
        assert rec[2:] == [0.0, 0.0]
        assert_close(h.norm(kind=kind, pre_scale=c)[0].item(), norm, tol, "no bound")
    assert all(torch.equal(a, b) for a, b in zip(before, t.host()))
    t.check_guards()
    h.close()


@gpu
def test_no_tensors_and_only_empty_ones():
    import torch
    for tensors in ([], [torch.empty(0, device="cuda")], [torch.empty(0, device="cuda", dtype=torch.bfloat16)] * 3):
        h = ar.Grads(tensors)
        per = torch.ones(max(1, len(tensors)), device="cuda")
        assert h.norm(max_norm=0.0, per_tensor=per).tolist() == [0.0, 1.0, 0.0, 0.0]
        assert h.clip(1.0, pre_scale=0.5).tolist() == [0.0, 0.5, 0.0, 0.0]
        assert per[:len(tensors)].tolist() == [0.0] * len(tensors)
        e = [torch.empty(0, device="cuda") for _ in tensors]
        ar.AdamW(e, tensors, e, e).step(1, lr=1e-3, clip=h.record)
        torch.cuda.synchronize()


# Values whose squares leave float32's range, alone and beside ordinary ones.
@gpu
@pytest.mark.parametrize("types", ["float32", "bfloat16"])
@pytest.mark.parametrize("size", [1, 33, 4099, 50021, 200003])
@pytest.mark.parametrize("values", ["huge", "top", "small", "subnormal", "zeros", "zeros-and-one", "huge-and-small",
                                    "edge", "steps"])
def test_norm_over_the_whole_range(values, size, types):
    import torch
    t = Tensors([size], types, offset=1, seed=5)
    v = t.views[0]
    x = v.double()
    if values == "huge":
        x = x * 1e30
    elif values == "top":
        x = torch.full_like(x, 3.3e38)
    elif values == "small":
        x = x * 1e-30
    elif values == "subnormal":
        x = torch.full_like(x, 1e-39)
    elif values in ("zeros", "zeros-and-one"):
        x = torch.zeros_like(x)
        if values == "zeros-and-one":
            x[size // 2] = -1.5
    elif values == "huge-and-small":
        x[::3] *= 1e25
        x[1::3] *= 1e-25
    elif values == "edge":
        x = torch.full_like(x, 2.0 ** -50)  # group sums around the bound of the float32 path
        x[::2] = 2.0 ** -52
    else:
        x = 2.0 ** (torch.arange(size, device="cuda").double() % 250 - 125)
    v.copy_(x.to(v.dtype))
    h = ar.Grads(t.views)
    norm, _ = true_norms(t.wide(), "l2", 1.0)
    rec = h.norm(max_norm=1.0).tolist()
    if norm > 3.4028235677973366e38:
        assert rec[0] == math.inf and rec[2] == 0.0 and rec[3] == 1.0
        assert_close(rec[1], 1.0 / norm, 11 * U, "scale")
    else:
        assert_close(rec[0], norm, 10 * U, values)
        assert rec[2:] == [0.0, float(norm > 1.0)]
    top = h.norm(kind="max").tolist()
    assert top[0] == float(v.double().abs().max()) and top[2] == 0.0
    h.close()


@gpu
@pytest.mark.parametrize("types", ["float32", "bfloat16"])
@pytest.mark.parametrize("rest", [[], [150001]])
@pytest.mark.parametrize("where", [0, 1, 20, 4500, 9000])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_nonfinite_gradients(bad, where, rest, types):
    import torch
    sizes = [300, 9001] + rest
    t = Tensors(sizes, types, offset=1)
    t.views[1][where] = bad
    before = t.host()
    h = ar.Grads(t.views)
    per = torch.empty(len(sizes), device="cuda")
    for kind in ("l2", "max"):
        rec = h.norm(max_norm=1.0, kind=kind, pre_scale=0.25, per_tensor=per).tolist()
        assert rec[1:] == [0.25, 1.0, 0.0]
        assert math.isnan(rec[0]) if math.isnan(bad) else rec[0] == math.inf
        assert [math.isfinite(x) for x in per.tolist()] == [True, False, True][:len(sizes)]
    p, m, v = (Tensors(sizes, "float32", seed=k, square=k == 3) for k in (1, 2, 3))
    kept = [x.host() for x in (p, m, v)]
    opt = ar.AdamW(p.views, t.views, m.views, v.views)
    opt.step(1, lr=1e-2, weight_decay=0.1, clip=h.record)
    for x, old in zip((p, m, v), kept):  # a skipped update leaves everything
        assert all(torch.equal(a, b) for a, b in zip(x.host(), old))
    # clipping scales by the pre-scale alone and leaves infinities and NaN
    assert h.clip(1.0, pre_scale=0.25).tolist()[1:] == [0.25, 1.0, 0.0]
    for a, b in zip(t.host(), before):
        assert torch.equal(a.nan_to_num(7.0), (b.float() * 0.25).to(b.dtype).nan_to_num(7.0))
    t.check_guards()


@gpu
@pytest.mark.parametrize("offsets", [(0, 0), (1, 1), (0, 1), (3, 2), (4, 0)])
@pytest.mark.parametrize("pair", [("float32", None), ("bfloat16", None), ("float32", "float32"),
                                  ("bfloat16", "float32"), ("float32", "bfloat16"), ("bfloat16", "bfloat16"),
                                  ("mixed", "float32")])
@pytest.mark.parametrize("sizes", ["tiny", "empties", "warp-edges", "item-edges", "ragged", "many"])
def test_clip(sizes, pair, offsets):
    import torch
    n = SIZES[sizes]
    g = Tensors(n, types_of(pair[0], len(n)), offsets[0], seed=3)
    o = None if pair[1] is None else Tensors(n, pair[1], offsets[1], seed=4)
    before, wide = g.host(), g.wide()
    norm, _ = true_norms(wide, "l2", 0.5)
    h = ar.Grads(g.views, out=None if o is None else o.views)
    rec = h.clip(0.25 * norm, pre_scale=0.5).tolist()
    assert_close(rec[0], norm, 10 * U, "norm")
    assert_close(rec[1], 0.125, 11 * U, "scale")
    assert rec[2:] == [0.0, 1.0]
    got = g if o is None else o
    for b, a in zip(before, got.host()):
        assert torch.equal(a, (b.float() * rec[1]).to(a.dtype))
    if o is not None:
        assert all(torch.equal(a, b) for a, b in zip(g.host(), before))
        o.check_guards()
    g.check_guards()
    # within the bound: in place nothing changes, elsewhere it is a copy
    before = g.host()
    rec = h.clip(1e9).tolist()
    assert rec[1:] == [1.0, 0.0, 0.0]
    for b, a in zip(before, got.host()):
        assert torch.equal(a, b.to(a.dtype))
    assert h.clip(0.0).tolist()[1:] == [0.0, 0.0, 1.0]  # a bound of zero
    assert all(not bool(a.any()) for a in got.host())
    h.close()


def adamw_reference(p, g, m, v, s, step, lr, b1, b2, eps, wd):
    """(new p, m, v and the three error bounds), in 64 bits."""
    g = g * s
    bc1, bc2 = 1.0 - b1 ** step, 1.0 - b2 ** step
    big = (b1 * m).abs() + ((1 - b1) * g).abs()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    den = (v / bc2).sqrt() + eps
    new = p * (1 - lr * wd) - lr / bc1 * m / den
    tiny = 2.0 ** -140  # sums of float32 subnormals
    pe = U * new.abs() + 16 * U * (lr / bc1 * big / den) + 3 * U * (lr * wd * p).abs() + tiny
    return new, m, v, pe, 6 * U * big + tiny, 8 * U * v + tiny


@gpu
@pytest.mark.parametrize("offsets", [(0, 0, 0, 0, 0), (0, 1, 0, 0, 0), (1, 1, 1, 1, 1), (2, 1, 0, 3, 5),
                                     (4, 4, 4, 4, 4)])
@pytest.mark.parametrize("kinds", [("float32", "float32", False), ("float32", "bfloat16", True),
                                   ("float32", "mixed", False), ("float32", "float32", True),
                                   ("bfloat16", "bfloat16", False), ("bfloat16", "float32", False),
                                   ("mixed", "mixed", False)])
@pytest.mark.parametrize("sizes", ["tiny", "empties", "warp-edges", "item-edges", "ragged", "many"])
def test_adamw(sizes, kinds, offsets):
    import torch
    n = SIZES[sizes]
    k = len(n)
    p = Tensors(n, types_of(kinds[0], k), offsets[0], seed=1, sigma=0.05)
    g = Tensors(n, types_of(kinds[1], k), offsets[1], seed=2, sigma=1e-2)
    m = Tensors(n, "float32", offsets[2], seed=3, sigma=3e-3)
    v = Tensors(n, "float32", offsets[3], seed=4, sigma=1e-2, square=True)
    w = Tensors(n, "bfloat16", offsets[4], seed=5) if kinds[2] else None
    decay = [float(i % 2) for i in range(k)]
    before = [x.wide() for x in (p, g, m, v)]
    grads = g.host()
    opt = ar.AdamW(p.views, g.views, m.views, v.views, copies=w.views if w else None, decay=decay)
    h = ar.Grads(g.views)
    record = h.norm(max_norm=1e-2)
    hyper = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8)
    opt.step(7, weight_decay=0.1, clip=record, **hyper)
    s = record[1].item()
    for i in range(k):
        want = adamw_reference(*[b[i] for b in before], s, 7, 3e-3, 0.9, 0.95, 1e-8, 0.1 * decay[i])
        for x, value, bound in ((p, want[0], want[3]), (m, want[1], want[4]), (v, want[2], want[5])):
            got = x.views[i].double().cpu()
            if x.views[i].dtype == torch.bfloat16:
                bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * value.abs()
            assert bool(((got - value).abs() <= bound).all()), (i, n[i])
        if w:
            assert torch.equal(w.views[i], p.views[i].bfloat16())
    assert all(torch.equal(a, b) for a, b in zip(grads, g.host()))
    for x in (p, g, m, v, w):
        if x:
            x.check_guards()


@gpu
def test_adamw_first_steps_and_edges():
    """Step 1 from zero moments moves every parameter by lr; betas of zero;
    gradients of zero change nothing but the decay; no record: factor 1."""
    import torch
    n = [1000, 3]
    g = Tensors(n, "float32", seed=2)
    z = [torch.zeros(k, device="cuda") for k in n]
    p, m, v = ([x.clone() for x in z] for _ in range(3))
    ar.AdamW(p, g.views, m, v).step(1, lr=0.5)
    for x, y in zip(p, g.views):
        assert bool(((x + 0.5 * y.sign()).abs() <= 1e-5).all())  # eps against |g|: at most 1e-8 / 1e-3
    p, m, v = ([x.clone() for x in z] for _ in range(3))
    ar.AdamW(p, g.views, m, v).step(1, lr=0.5, beta1=0.0, beta2=0.0)
    for x, y, a, b in zip(p, g.views, m, v):
        assert torch.equal(a, y) and torch.equal(b, y * y)
    p = [torch.ones_like(x) for x in z]
    m, v = ([x.clone() for x in z] for _ in range(2))
    opt = ar.AdamW(p, [x.clone() for x in z], m, v)
    for t in range(1, 4):
        opt.step(t, lr=0.25, weight_decay=0.5)
    assert all(bool((x == 0.875 ** 3).all()) for x in p) and not any(bool(x.any()) for x in m + v)
    opt.step(10 ** 12, lr=0.0)
    assert all(bool((x == 0.875 ** 3).all()) for x in p)


@gpu
def test_adamw_counts_its_updates_on_the_device():
    """The counted form gives what the host's numbers give, in a graph too,
    reads its rate when it runs, and does not count a skipped update."""
    import torch
    n = [4099, 3]
    g = Tensors(n, "float32", seed=2, sigma=1e-2)
    a = [Tensors(n, "float32", seed=1) for _ in range(2)]
    m, v = ([[torch.zeros(k, device="cuda") for k in n] for _ in range(2)] for _ in range(2))
    host, device = (ar.AdamW(a[i].views, g.views, m[i], v[i]) for i in range(2))
    steps, lr = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.full((1,), 0.125, device="cuda")
    record = torch.tensor([1.0, 0.5, 0.0, 1.0], device="cuda")
    device.step(steps, lr=lr, weight_decay=0.25, clip=record)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        device.step(steps, lr=lr, weight_decay=0.25, clip=record)
    rates = [0.125, 0.5, 0.25, 0.0625]
    for t in range(1, 5):
        if t > 1:
            lr.fill_(rates[t - 1])
            graph.replay()
        host.step(t, lr=rates[t - 1], weight_decay=0.25, clip=record)
        assert steps.item() == t
        for i in range(2):
            assert torch.equal(m[0][i], m[1][i]) and torch.equal(v[0][i], v[1][i])
            # the two scalars may round apart by one float32 unit: 4 u of an update
            x, y = a[0].views[i], a[1].views[i]
            assert bool(((x - y).abs() <= 8 * U * (x.abs() + rates[t - 1] * 10)).all())
            y.copy_(x)
    kept = a[1].host()
    record[2] = 1.0
    graph.replay()
    assert steps.item() == 4 and all(torch.equal(x, y) for x, y in zip(kept, a[1].host()))
    steps.fill_(10 ** 15)
    record[2] = 0.0
    device.step(steps, lr=0.0, clip=record)
    assert steps.item() == 10 ** 15 + 1 and all(torch.equal(x, y) for x, y in zip(kept, a[1].host()))
    with pytest.raises(ValueError, match="one int64"):
        device.step(steps.int(), lr=0.1)
    with pytest.raises(ValueError, match="lr"):
        device.step(steps, lr=lr.double())
    with pytest.raises(ar.ArError):
        device.step(steps, lr=-1.0)
    L, p = ar.lib(), ar.AdamWParams(0, 0.1, 0.9, 0.99, 1e-8, 0.0)
    for bad in (None, steps.data_ptr() + 4, torch.zeros(1, dtype=torch.int64).data_ptr()):
        assert L.ar_adamw_step_counted(device._h, ctypes.byref(p), bad, None, None, None) == 1
    assert steps.item() == 10 ** 15 + 1


@gpu
def test_dense_tensors_in_another_order():
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    base = [torch.randn(48, 33, generator=g, device="cuda") for _ in range(4)]
    p, gr, m, v = ([base[i].t()] for i in range(4))
    v[0].square_()
    want = adamw_reference(*[x[0].double().cpu() for x in (p, gr, m, v)], 1.0, 2, 1e-2, 0.9, 0.99, 1e-8, 0.0)
    ar.AdamW(p, gr, m, v).step(2, lr=1e-2, beta2=0.99)
    assert bool(((p[0].double().cpu() - want[0]).abs() <= want[3]).all())
    h = ar.Grads(gr, out=[torch.empty(48, 33, device="cuda").t()])
    rec = h.clip(1.0).tolist()
    assert torch.equal(h.out[0], gr[0] * rec[1])
    with pytest.raises(ValueError, match="another order"):
        ar.Grads(gr, out=[torch.empty(33, 48, device="cuda")])
    with pytest.raises(ValueError, match="not dense"):
        ar.Grads([base[0][:, ::2]])


@gpu
def test_calls_repeat_bit_for_bit_on_any_stream_and_in_graphs():
    import torch
    t = Tensors([1000003, 7, 65537], types_of("mixed", 3), offset=1, seed=9)
    out = Tensors([1000003, 7, 65537], "float32", offset=1)
    h = ar.Grads(t.views, out=out.views)
    first = h.clip(0.5).clone()
    ref = out.host()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for k in range(5):
        for v in out.views:
            v.zero_()
        s.wait_stream(torch.cuda.current_stream())
        rec = torch.empty(4, device="cuda")
        h.clip(0.5, result=rec, stream=s)
        s.synchronize()
        assert torch.equal(rec, first) and all(torch.equal(a, b) for a, b in zip(ref, out.host()))
    graph = torch.cuda.CUDAGraph()
    rec = torch.zeros(4, device="cuda")
    p, m, v = (Tensors([1000003, 7, 65537], "float32", seed=k, square=k == 3) for k in (1, 2, 3))
    opt = ar.AdamW(p.views, t.views, m.views, v.views)
    opt.step(1, lr=0.0)  # moments alone, before the capture
    start = [x.host() for x in (p, m, v)]
    with torch.cuda.graph(graph):
        h.clip(0.5, result=rec)
        opt.step(2, lr=1e-3, clip=rec)
    for k in range(2):
        for x, old in zip((p, m, v), start):
            for a, b in zip(x.views, old):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(rec, first) and all(torch.equal(a, b) for a, b in zip(ref, out.host()))
        state = [x.host() for x in (p, m, v)]
        if k:
            assert all(torch.equal(a, b) for x, y in zip(state, kept) for a, b in zip(x, y))  # noqa: F821
        kept = state  # noqa: F841


@gpu
def test_offsets_past_32_bits():
    """One tensor of more than 2^32 elements: every element counts, the last
    ones are reached."""
    import torch
    n = (1 << 32) + 4099
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough free device memory")
    x = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    h = ar.Grads([x])
    rec = h.norm(max_norm=1.0).tolist()
    assert_close(rec[0], 0.5 * math.sqrt(n), U, "norm")  # group sums are exact here
    x[n - 1] = 1024.0
    assert h.norm(kind="max")[0].item() == 1024.0
    x[n - 1] = 0.5
    rec = h.clip(0.25 * math.sqrt(n)).tolist()
    for at in (0, (1 << 31) - 4, (1 << 32) - 4, n - 8):
        assert bool((x[at:at + 8] == 0.25).all())
    assert float(x.max()) == 0.25 and float(x.min()) == 0.25
    h.close()
    del x, h
    n = (1 << 31) + 4099
    p, g = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.ones(n, dtype=torch.bfloat16, device="cuda")
    m, v = (torch.zeros(n, device="cuda") for _ in range(2))
    g[n - 1] = -1.0
    ar.AdamW([p], [g], [m], [v]).step(1, lr=0.5)  # the first update moves by lr, eps and roundings aside
    assert float(p[:n - 1].max()) == -0.5 and float(p[:n - 1].min()) == -0.5 and p[n - 1].item() == 0.5
    assert bool((v == v[0]).all()) and bool((m[:n - 1] == m[0]).all()) and m[n - 1].item() == -m[0].item() != 0.0


@gpu
@pytest.mark.parametrize("types", ["float32", "bfloat16"])
def test_sets_around_the_kernels_limits(types):
    """Ranges on both sides of one cluster (128), of one wave of warps (3648),
    and enough that warps draw them: the sums, and each tensor's own."""
    import torch
    wave = 152 * 3 * 8
    for n in ([1] * 127, [1] * 128, [1] * 129, [1024] * 128, [1023, 1025] * 64, [5] * wave, [5] * (wave + 1),
              [3] * (9 * wave), [wave * 1024 - 1], [wave * 1024], [wave * 12288 + 7, 11], [3 * wave * 12288, 1, 70000]):
        x = torch.empty(sum(n), dtype=tdt(types), device="cuda")
        x.copy_(torch.randn(x.numel(), generator=torch.Generator(device="cuda").manual_seed(len(n)), device="cuda"))
        h = ar.Grads(list(x.split(n)))
        wide = x.double().square_()
        each = [c.sum() for c in wide.split(n)] if len(n) < 1000 else list(wide.view(len(n), -1).sum(1))
        per = torch.empty(len(n), device="cuda")
        for k in range(2):  # the counters are back in place
            got = h.norm(per_tensor=per)[0].item()
            assert_close(got, math.sqrt(wide.sum().item()), 10 * U, (len(n), n[0]))
            want = torch.stack(each).sqrt()
            assert bool(((per.double() - want).abs() <= 10 * U * want).all())
        rec = h.clip(0.5 * got).tolist()
        assert_close(rec[1], 0.5, 12 * U, "scale")
        h.close()


@gpu
@pytest.mark.parametrize("P,n", [(1, 1000), (3, 100003), (8, 70), (8, 1000001)])
def test_sharded_training_step(P, n):
    """reduce-scatter, norm, AdamW, all-gather: the norm is the averaged
    gradient's, every rank ends with the owners' rounded weights, and the loss
    falls."""
    import sys
    import torch
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import zero_step
    z = zero_step.ZeroStep(P, n, weight_decay=0.01)
    chunks = zero_step.owned(P, n)
    assert sorted(i for a, b in chunks for i in range(a, b)) == list(range(n))
    losses = []
    for _ in range(4):
        losses.append(z.backward().item())
        mean = sum(g.double() for g in z.grads) / P
        before = [x.double().cpu() for x in z.master], [x.double().cpu() for x in z.exp_avg], \
            [x.double().cpu() for x in z.exp_avg_sq]
        rec = z.step().tolist()
        # P - 1 float32 additions and a division: P u of the terms' magnitudes, below 2 P u of a norm of this kind
        assert_close(rec[0], float(mean.norm()), (10 + 2 * P) * U, "norm")
        for r, (a, b) in enumerate(chunks):
            g = z.grads[r][a:b].double().cpu()
            want = adamw_reference(before[0][r], g, before[1][r], before[2][r], rec[1], z.steps.item(), z.lr, 0.9,
                                   0.999, 1e-8, 0.01)
            assert bool(((z.master[r].double().cpu() - want[0]).abs() <= want[3]).all())
            assert all(torch.equal(w[a:b], z.master[r].bfloat16()) for w in z.weights)
    assert losses == sorted(losses, reverse=True)
    z.scatter.check()
    z.gather.check()
    graph = z.capture()
    for _ in range(3):
        losses.append(z.backward().item())
        graph.replay()
        assert all(torch.equal(z.weights[0], w) for w in z.weights)
    assert losses == sorted(losses, reverse=True) and z.steps.item() == 7


@gpu
def test_refusals():
    import torch
    a, b = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    h = ar.Grads([a, b])

    def status(f, *args, **kw):
        with pytest.raises(ar.ArError) as e:
            f(*args, **kw)
        return e.value.name
    bad = "AR_ERR_INVALID_ARG"
    for kw in ({"pre_scale": 0.0}, {"pre_scale": -1.0}, {"pre_scale": math.nan}, {"pre_scale": math.inf},
               {"pre_scale": 1e-40}, {"max_norm": -1.0}, {"max_norm": math.nan}):
        assert status(h.norm, **kw) == bad
    with pytest.raises(KeyError):
        h.norm(kind="l3")
    with pytest.raises(ValueError, match="result"):
        h.norm(result=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError, match="result"):
        h.norm(result=torch.zeros(4))
    with pytest.raises(ValueError, match="per_tensor"):
        h.norm(per_tensor=torch.zeros(1, device="cuda"))
    L = ar.lib()
    host = torch.zeros(4)
    assert L.ar_grad_norm(h._h, 0, 1.0, 1.0, host.data_ptr(), None, None) == 1
    assert L.ar_grad_norm(h._h, 0, 1.0, 1.0, None, None, None) == 1
    assert L.ar_grad_norm(h._h, 0, 1.0, 1.0, a.data_ptr() + 2, None, None) == 1
    assert L.ar_grad_norm(h._h, 2, 1.0, 1.0, a.data_ptr(), None, None) == 1
    # tensors that overlap, in the list and across lists
    assert status(ar.Grads, [a, a]) == bad
    assert status(ar.Grads, [a[:40], a[30:]]) == bad
    assert status(ar.Grads, [a], out=[a.view(torch.bfloat16)[:64]]) == bad
    assert status(ar.Grads, [a[:40], b], out=[b[:40], torch.zeros(64, device="cuda")]) == bad
    assert status(ar.AdamW, [a], [b], [torch.zeros(64, device="cuda")], [b]) == bad
    with pytest.raises(ValueError, match="expected 2 tensors"):
        ar.Grads([a, b], out=[a])
    with pytest.raises(ValueError, match="expected 64 elements"):
        ar.Grads([a], out=[b[:63]])
    # through the C ABI: host memory, a tensor longer than its allocation, a pointer off its alignment
    one, f32 = (ctypes.c_uint64 * 1)(4), (ctypes.c_int * 1)(1)

    def create(ptr, count=one):
        out = ctypes.c_void_p()
        return L.ar_grads_create(1, count, f32, (ctypes.c_void_p * 1)(ptr), None, None, ctypes.byref(out))
    assert create(host.data_ptr()) == 1 and create(None) == 1 and create(a.data_ptr() + 1) == 1
    assert create(a.data_ptr(), (ctypes.c_uint64 * 1)(1 << 38)) == 1
    c, d = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    opt = ar.AdamW([a], [b], [c], [d])
    for kw in ({"lr": -1.0}, {"lr": math.nan}, {"lr": 1.0, "beta1": 1.0}, {"lr": 1.0, "beta2": -0.1},
               {"lr": 1.0, "eps": 0.0}, {"lr": 1.0, "eps": 1e-40}, {"lr": 1.0, "weight_decay": -0.1},
               {"lr": 1.0, "weight_decay": math.inf}, {"lr": 3e38, "beta1": 0.9}):
        assert status(opt.step, 1, **kw) == bad
    with pytest.raises(ValueError, match="step"):
        opt.step(0, lr=1.0)
    with pytest.raises(ValueError, match="clip"):
        opt.step(1, lr=1.0, clip=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError, match="element type"):
        ar.AdamW([a], [b], [c.bfloat16()], [d])
    with pytest.raises(ValueError, match="decay"):
        ar.AdamW([a], [b], [c], [d], decay=[1.0, 1.0])
    assert status(ar.AdamW, [a], [b], [c], [d], decay=[-1.0]) == bad
    assert status(ar.AdamW, [a.bfloat16()], [b], [c], [d], copies=[a.bfloat16()]) == bad
    torch.cuda.synchronize()
    assert not any(bool(x.any()) for x in (a, b, c, d))
