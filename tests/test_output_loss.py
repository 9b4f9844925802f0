"""The output layer's losses and gradients, against their definitions in 64 bits.

Tolerances, derived from the arithmetic and not from its output.  u = 2^-24.

* A product of two bf16 values is exact in float32.  A sum of k products in any
  order, each addition rounded or cut off (2 u relative to the partial sum), is
  off by at most 2 u (k + 4) sum |a b|; call it S(k) sum |a b|.  float32 operands
  are three bf16 planes and six products a term: what they leave out and the
  splits are below 4 u |a b|, the additions six times as many: S(6 k) + 4 u.
* Logits of temperature t: e = S(D) sum |x w| / t off.  In the softmax the scaling
  by log2(e) / t and the subtraction of the largest round twice (4 u |z / t|), ex2
  is off by 2^-22 relative, sums of V positive terms in float32 by S(V) at most: q's
  relative error is d = 2 e + 8 u (|z / t| + 2) + S(V) + 16 u, e and |z / t| their
  largest in the row.
* The teacher's shares: the product with 1 / t and the difference round (4 u of the
  largest difference), exp 2 ulp, sum and quotient: s = 4 u |diff| + S(k) + 16 u.
* Loss: t^2 (2 d + s (|log p| + |z / t| + 2) + 4 u (|loss| / t^2)).
* Gradient of the logits: f t (q d + p (s + 4 u)), and in bf16 one rounding: 2^-8 |g|.
* Gradients: the sums over what each logit gradient may be off, S of their own
  sums, and one rounding to the result's type: 2^-8 or u relative.
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

@pytest.mark.parametrize("tokens, vocab, piece", [(0, 1, 0), (1, 255, 0), (256, 256, 0), (257, 7, 256), (1003, 300, 300),
                                                  (8192, 128000, 0), (1 << 22, 1 << 20, 0), (1 << 20, 1000003, 0)])
def test_pieces_tile_the_tokens(tokens, vocab, piece):
    info = ar.output_loss_layout(tokens, 64, vocab, piece=piece)
    rows, wide = max(256, -(-tokens // 256) * 256), -(-vocab // 256) * 256
    assert info["tiling_ok"] == 1 and info["piece"] % 256 == 0
    assert info["piece"] * info["pieces"] >= rows > info["piece"] * (info["pieces"] - 1)
    assert info["piece"] <= (-(-piece // 256) * 256 if piece else max(256, (1 << 28) // wide))
    assert info["workspace_bytes"] >= 6 * info["piece"] * wide
    less = ar.output_loss_layout(tokens, 64, vocab, piece=piece, grads=False)
    assert less["pieces"] == 1
    if info["pieces"] == 1:
        assert less["workspace_bytes"] <= info["workspace_bytes"] - 6 * info["piece"] * wide


def test_layout_refusals():
    def status(*a, **k):
        with pytest.raises(ar.ArError) as e:
            ar.output_loss_layout(*a, **k)
        return e.value.name
    assert status(4, 0, 8) == "AR_ERR_INVALID_ARG"
    assert status(4, 8, 0) == "AR_ERR_INVALID_ARG"
    assert status(4, 8, 8, top=-1) == "AR_ERR_INVALID_ARG"
    assert status(4, 8, 8, "int32") == "AR_ERR_UNSUPPORTED"
    assert status((1 << 22) + 1, 8, 8) == "AR_ERR_UNSUPPORTED"
    assert status(4, (1 << 16) + 1, 8) == "AR_ERR_UNSUPPORTED"
    assert status(4, 8, (1 << 24) + 1) == "AR_ERR_UNSUPPORTED"
    assert status(4, 8, 8, top=1025) == "AR_ERR_UNSUPPORTED"
    assert status(1 << 22, 8, 8, top=1024) == "AR_ERR_UNSUPPORTED"
    L, info = ar.lib(), ar.OutputLossInfo()
    assert L.ar_output_loss_layout(4, 8, 8, 9, 0, 0, 1, ctypes.byref(info)) == 1
    assert L.ar_output_loss_layout(4, 8, 8, 2, 0, 0, 1, None) == 1


def test_null_handles_are_refused():
    L, a, info = ar.lib(), ar.OutputLossArgs(), ar.OutputLossInfo()
    assert L.ar_output_loss_query(None, ctypes.byref(info)) == 1
    assert L.ar_output_loss_destroy(None) == 1
    assert L.ar_output_loss_check(None) == 1
    assert L.ar_output_loss_create(4, 8, 8, 2, 0, 0, 1, None) == 1
    assert L.ar_output_cross_entropy(None, ctypes.byref(a), None, 8, -100, None) == 1
    assert L.ar_output_distill(None, ctypes.byref(a), None, 8, 1, None, 1, 1, 1, 1.0, None) == 1


def test_matrices_the_binding_refuses():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        ar._rows_of(torch.zeros(3, 4), "x", 3, 4, ("float32",))
    with pytest.raises(ValueError, match="element type"):
        ar._rows_of(torch.zeros(3, 4), "x", 3, 4, ("bfloat16",))


# --------------------------------------------------------------------- on a GPU

def tdt(name):
    import torch
    return getattr(torch, name)


def half_step(name):
    return 2.0 ** -8 if name == "bfloat16" else U


def bound_of_sum(k, dtype):
    """S(k), with float32's splits."""
    return 2 * U * (k + 4) if dtype == "bfloat16" else 2 * U * (6 * k + 4) + 4 * U


class Expected:
    """The definition in 64 bits (on the host unless told), and how far float32
    may be off."""

    def __init__(self, x, w, ids, shares, t=1.0, scale=1.0, reduction="mean", dtype="bfloat16", spread=None, on="cpu"):
        """ids: lists of each token (empty: does not count); shares likewise;
        spread: the largest teacher difference / t of each token."""
        import torch
        x, w = x.double().to(on), w.double().to(on)
        self.on = on
        n, v = x.shape[0], w.shape[0]
        keep = [i for i in range(n) if ids[i]]
        self.counted = len(keep)
        self.factor = scale / max(1, len(keep)) if reduction == "mean" else scale
        p = torch.zeros(n, v, dtype=torch.float64, device=on)
        for i in keep:
            for j, s in zip(ids[i], shares[i]):
                p[i, j] += s
        mask = torch.zeros(n, 1, dtype=torch.float64, device=on)
        mask[keep] = 1.0
        xs = torch.where(mask > 0, x, 0.0)
        zt = xs @ w.t() / t
        logq = torch.log_softmax(zt, 1)
        q = logq.exp()
        plogp = torch.xlogy(p, p)
        self.losses = (t * t * (plogp - p * logq).sum(1)) * mask[:, 0]
        self.loss = math.fsum(self.losses.tolist()) * self.factor
        g = self.factor * t * (q - p) * mask
        self.dx, self.dw = g @ w, g.t() @ xs
        # what float32 may be off
        big = zt.abs().amax(1, keepdim=True)
        e = bound_of_sum(x.shape[1], dtype) * (xs.abs() @ w.abs().t()).amax(1, keepdim=True) / t
        d = 2 * e + 8 * U * (big + 2) + 2 * U * (v + 4) + 16 * U
        longest = max([1] + [len(i) for i in ids])
        s = 0.0 if spread is None else 4 * U * spread.double().reshape(-1, 1) + 2 * U * (longest + 4) + 16 * U
        logp = torch.where(p > 0, -p.clamp(min=1e-300).log(), 0.0).amax(1, keepdim=True)
        self.losses_tol = (t * t * (2 * d + s * (logp + big + 2)) * mask)[:, 0] + 4 * U * self.losses.abs()
        self.loss_tol = float(self.losses_tol.sum()) * self.factor + 4 * U * abs(self.loss)
        g_tol = self.factor * t * (q * d + p * (s + 4 * U)) * mask + half_step(dtype) * g.abs()
        sv, sn = bound_of_sum(v, dtype), bound_of_sum(n, dtype)
        self.dx_tol = g_tol @ w.abs() + sv * (g.abs() @ w.abs())
        self.dw_tol = g_tol.t() @ xs.abs() + sn * (g.abs().t() @ xs.abs())

    def check(self, record, losses=None, dx=None, dw=None, x0=None, w0=None):
        """x0, w0: what the gradients were added to."""
        loss, counted, nonfinite, factor = record.tolist()
        assert counted == self.counted and nonfinite == 0.0
        assert factor == pytest.approx(self.factor, rel=2 * U)
        assert abs(loss - self.loss) <= self.loss_tol + 1e-40
        if losses is not None:
            assert bool(((losses.double().to(self.on) - self.losses).abs() <= self.losses_tol).all())
        for got, want, tol, old in ((dx, self.dx, self.dx_tol, x0), (dw, self.dw, self.dw_tol, w0)):
            if got is None:
                continue
            h = half_step(str(got.dtype).replace("torch.", ""))
            if old is not None:
                want = want + old.double().to(self.on)
            off = (got.double().to(self.on) - want).abs()
            room = tol * (1 + 2 * h) + 2 * h * want.abs() + 1e-38  # the sum with what was there rounds in float32 too
            assert bool((off <= room).all()), float((off / room).max())


def make(n, d, v, dtype, seed=0, gain=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, d, generator=g).to(tdt(dtype)).cuda()
    w = (torch.randn(v, d, generator=g) * (gain * 1.3 / math.sqrt(d))).to(tdt(dtype)).cuda()
    return x, w, g


def targets_of(n, v, g, keep=1.0):
    import torch
    t = torch.randint(v, (n,), generator=g)
    if keep < 1.0:
        t[torch.rand(n, generator=g) >= keep] = -100
    return t


def one_hot_lists(targets):
    ids = [[int(t)] if t != -100 else [] for t in targets.tolist()]
    return ids, [[1.0] * len(i) for i in ids]


def run_ce(h, x, w, targets, dtype, grads=("hidden", "weight"), gtype=None, **more):
    import torch
    gt = tdt(gtype or dtype)
    dx = torch.full(x.shape, 7.0, dtype=gt, device="cuda") if "hidden" in grads else None
    dw = torch.full(w.shape, 7.0, dtype=gt, device="cuda") if "weight" in grads else None
    losses = torch.full((x.shape[0],), 7.0, device="cuda")
    rec = h.cross_entropy(x, w, targets.cuda(), grad_hidden=dx, grad_weight=dw, losses=losses, **more)
    h.check()
    return rec.clone(), losses, dx, dw


SIZES = [(1, 1, 1), (1, 8, 2), (3, 5, 7), (37, 129, 203), (255, 64, 256), (256, 64, 257), (257, 72, 511),
         (300, 515, 1003), (513, 96, 2003), (129, 640, 130), (40, 1, 1), (300, 2, 70), (26, 7, 300)]


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n, d, v", SIZES)
@pytest.mark.parametrize("keep", [1.0, 0.6])
def test_cross_entropy(n, d, v, dtype, keep):
    x, w, g = make(n, d, v, dtype, seed=n + v)
    t = targets_of(n, v, g, keep)
    h = ar.OutputLoss(n, d, v, dtype)
    Expected(x, w, *one_hot_lists(t), dtype=dtype).check(*run_ce(h, x, w, t, dtype))


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n, d, v", [(1, 1, 65), (2, 1030, 300), (3, 515, 64), (4, 2050, 63), (5, 33, 1), (6, 640, 1003),
                                     (7, 129, 2003), (8, 4097, 130), (9, 4097, 130), (12, 1100, 2003)])
@pytest.mark.parametrize("keep", [1.0, 0.5])
def test_few_tokens(n, d, v, dtype, keep):
    """Calls of a few tokens take kernels of their own (float32 in groups of eight),
    also on odd and accumulating rows, with lists and in float32 results."""
    import torch
    x, w, g = make(n, d, v, dtype, seed=n * d)
    t = targets_of(n, v, g, keep)
    h = ar.OutputLoss(20, d, v, dtype, top=5)
    Expected(x, w, *one_hot_lists(t), dtype=dtype).check(*run_ce(h, x, w, t, dtype))
    want = Expected(x, w, *one_hot_lists(t), reduction="sum", scale=1.0 / 300, dtype=dtype)
    want.check(*run_ce(h, x, w, t, dtype, gtype="float32", reduction="sum", scale=1.0 / 300))
    for grads in ((), ("hidden",), ("weight",)):
        want.check(*run_ce(h, x, w, t, dtype, grads, reduction="sum", scale=1.0 / 300))
    k = min(5, v)
    ids, logits = teacher(n, k, v, g, dtype, 0.4, twice=True)
    lists, shares, spread = teacher_lists(ids, logits, 2.0)
    big = torch.zeros(n, d + 3, dtype=x.dtype, device="cuda")
    big[:, 1:-2] = x
    dx = torch.ones(n, d + 1, dtype=x.dtype, device="cuda")[:, 1:]
    dw = (0.01 * torch.randn(v, d, generator=g)).to(tdt(dtype)).cuda()
    x0, w0 = dx.clone(), dw.clone()
    rec = h.distill(big[:, 1:-2], w, ids.cuda(), logits.cuda(), temperature=2.0, grad_hidden=dx, grad_weight=dw,
                    accumulate=True)
    Expected(x, w, lists, shares, 2.0, dtype=dtype, spread=spread).check(rec, None, dx, dw, x0, w0)


@gpu
@pytest.mark.parametrize("keep", [1.0, 0.3])
def test_few_tokens_of_large_float32_weights(keep):
    x, w, g = make(21, 4100, 4100, "float32", seed=7)
    t = targets_of(21, 4100, g, keep)
    h = ar.OutputLoss(21, 4100, 4100, "float32")
    want = Expected(x, w, *one_hot_lists(t), dtype="float32")
    want.check(*run_ce(h, x, w, t, "float32"))
    want.check(*run_ce(h, x, w, t, "float32", ()))


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n, d, v, piece", [(700, 40, 303, 256), (1100, 136, 500, 512), (257, 1000, 77, 256)])
def test_pieces(n, d, v, piece, dtype):
    x, w, g = make(n, d, v, dtype, seed=3)
    t = targets_of(n, v, g, 0.8)
    h = ar.OutputLoss(n, d, v, dtype, piece=piece)
    assert h.info()["pieces"] > 1
    want = Expected(x, w, *one_hot_lists(t), reduction="sum", scale=0.25, dtype=dtype)
    want.check(*run_ce(h, x, w, t.int(), dtype, reduction="sum", scale=0.25))


@gpu
@pytest.mark.parametrize("dtype, gtype", [("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float32", "float32")])
@pytest.mark.parametrize("n, d, v", [(1700, 40, 303), (2400, 270, 130)])
@pytest.mark.parametrize("keep", [1.0, 0.3])
def test_more_pieces_than_are_kept(n, d, v, keep, dtype, gtype):
    """The weights' gradient is summed in memory over several runs of pieces; the
    last ones may hold no token that counts."""
    import torch
    x, w, g = make(n, d, v, dtype, seed=25)
    t = targets_of(n, v, g, keep)
    h = ar.OutputLoss(n, d, v, dtype, piece=256)
    assert h.info()["pieces"] > 4
    want = Expected(x, w, *one_hot_lists(t), dtype=dtype)
    want.check(*run_ce(h, x, w, t, dtype, gtype=gtype))
    dx, dw = (0.01 * torch.randn(a.shape, generator=g).to(tdt(gtype)).cuda() for a in (x, w))
    x0, w0 = dx.clone(), dw.clone()
    rec = h.cross_entropy(x, w, t.cuda(), grad_hidden=dx, grad_weight=dw, accumulate=True)
    want.check(rec, None, dx, dw, x0, w0)


@gpu
@pytest.mark.parametrize("grads", [(), ("hidden",), ("weight",)])
@pytest.mark.parametrize("piece", [0, 256])
def test_one_gradient_or_none(grads, piece):
    x, w, g = make(390, 72, 600, "bfloat16", seed=4)
    t = targets_of(390, 600, g, 0.7)
    h = ar.OutputLoss(390, 72, 600, piece=piece, grads=bool(grads))
    Expected(x, w, *one_hot_lists(t)).check(*run_ce(h, x, w, t, "bfloat16", grads))


@gpu
def test_gradients_in_float32_of_bf16_inputs():
    x, w, g = make(530, 72, 700, "bfloat16", seed=5)
    t = targets_of(530, 700, g, 0.9)
    for piece in (0, 256):
        h = ar.OutputLoss(530, 72, 700, piece=piece)
        Expected(x, w, *one_hot_lists(t)).check(*run_ce(h, x, w, t, "bfloat16", gtype="float32"))


@gpu
@pytest.mark.parametrize("gtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("piece", [0, 256])
def test_gradients_are_added(gtype, piece):
    import torch
    x, w, g = make(630, 72, 300, "bfloat16", seed=6)
    t = targets_of(630, 300, g, 0.5)
    h = ar.OutputLoss(630, 72, 300, piece=piece)
    dx = (0.01 * torch.randn(x.shape, generator=g)).to(tdt(gtype)).cuda()
    dw = (0.01 * torch.randn(w.shape, generator=g)).to(tdt(gtype)).cuda()
    x0, w0 = dx.clone(), dw.clone()
    rec = h.cross_entropy(x, w, t.cuda(), grad_hidden=dx, grad_weight=dw, accumulate=True)
    Expected(x, w, *one_hot_lists(t)).check(rec, None, dx, dw, x0, w0)
    ignored = (t == -100).cuda()
    assert torch.equal(dx[ignored], x0[ignored])


def teacher(n, k, v, g, dtype, absent=0.0, twice=False):
    """ids (distinct unless `twice`), logits; entries absent by id or by -infinity."""
    import torch
    ids = torch.stack([torch.randperm(v, generator=g)[:k] for _ in range(n)])
    if twice and k > 1:
        ids[:, k // 2] = ids[:, 0]
        ids[:, -1] = ids[:, 0]
    logits = (4.0 * torch.randn(n, k, generator=g)).to(tdt(dtype))
    if absent:
        ids[torch.rand(n, k, generator=g) < absent / 2] = -1
        logits[torch.rand(n, k, generator=g) < absent / 2] = -math.inf
    return ids, logits


def teacher_lists(ids, logits, t):
    import torch
    out, shares, spread = [], [], torch.zeros(ids.shape[0])
    for i in range(ids.shape[0]):
        u = logits[i].double() / t
        there = [j for j in range(ids.shape[1]) if ids[i, j] >= 0 and u[j] != -math.inf]
        p = torch.softmax(u[there], 0) if there else u[:0]
        out.append([int(ids[i, j]) for j in there])
        shares.append(p.tolist())
        if there:
            spread[i] = u[there].max() - u[there].min()
    return out, shares, spread


def run_distill(h, x, w, ids, logits, dtype, **more):
    import torch
    dx, dw = torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda"), torch.full(w.shape, 7.0, dtype=w.dtype, device="cuda")
    losses = torch.full((x.shape[0],), 7.0, device="cuda")
    rec = h.distill(x, w, ids.cuda(), logits.cuda(), grad_hidden=dx, grad_weight=dw, losses=losses, **more)
    h.check()
    return rec.clone(), losses, dx, dw


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n, d, v, k, t", [(1, 8, 5, 1, 1.0), (5, 192, 400, 8, 1.0), (70, 129, 1003, 33, 2.0),
                                           (257, 64, 300, 300, 4.0), (300, 256, 2003, 64, 0.5), (40, 24, 1200, 1024, 1.0)])
@pytest.mark.parametrize("absent", [0.0, 0.6])
def test_distillation(n, d, v, k, t, dtype, absent):
    x, w, g = make(n, d, v, dtype, seed=k)
    ids, logits = teacher(n, k, v, g, dtype, absent)
    h = ar.OutputLoss(n, d, v, dtype, top=k)
    lists, shares, spread = teacher_lists(ids, logits, t)
    want = Expected(x, w, lists, shares, t, dtype=dtype, spread=spread)
    want.check(*run_distill(h, x, w, ids, logits, dtype, temperature=t))


@gpu
@pytest.mark.parametrize("k", [2, 31, 70])
def test_entries_of_one_id_add_up(k):
    x, w, g = make(50, 40, 600, "bfloat16", seed=8)
    ids, logits = teacher(50, k, 600, g, "float32", 0.2, twice=True)
    h = ar.OutputLoss(600, 40, 600, top=80, piece=256)
    lists, shares, spread = teacher_lists(ids, logits, 2.0)
    want = Expected(x, w, lists, shares, 2.0, spread=spread, reduction="sum", scale=3.0)
    want.check(*run_distill(h, x, w, ids.int(), logits, "bfloat16", temperature=2.0, reduction="sum", scale=3.0))


@gpu
def test_teacher_logits_of_absent_entries_are_not_looked_at():
    x, w, g = make(20, 40, 300, "bfloat16", seed=9)
    ids, logits = teacher(20, 6, 300, g, "bfloat16")
    ids[:, 3], ids[4] = -1, -7
    lists, shares, spread = teacher_lists(ids, logits, 1.0)
    logits[:, 3], logits[4] = math.nan, math.inf
    h = ar.OutputLoss(20, 40, 300, top=6)
    want = Expected(x, w, lists, shares, spread=spread)
    assert want.counted == 19
    want.check(*run_distill(h, x, w, ids, logits, "bfloat16"))


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n, d, v", [(300, 40, 300), (70, 515, 1003)])
def test_hidden_states_of_tokens_that_do_not_count_are_not_read(n, d, v, dtype):
    import torch
    x, w, g = make(n, d, v, dtype, seed=10)
    t = targets_of(n, v, g, 0.5)
    clean = x.clone()
    bad = torch.tensor([math.nan, math.inf, -math.inf])
    for i in (t == -100).nonzero()[:, 0].tolist():
        x[i] = bad[i % 3]
    h = ar.OutputLoss(n, d, v, dtype)
    rec, losses, dx, dw = run_ce(h, x, w, t, dtype)
    Expected(clean, w, *one_hot_lists(t), dtype=dtype).check(rec, losses, dx, dw)
    assert bool((losses[(t == -100).cuda()] == 0).all()) and bool((dx[(t == -100).cuda()] == 0).all())


@gpu
@pytest.mark.parametrize("piece", [0, 256])
def test_nothing_counts(piece):
    import torch
    x, w, _ = make(265, 40, 600, "bfloat16")
    h = ar.OutputLoss(265, 40, 600, top=3, piece=piece)
    rec, losses, dx, dw = run_ce(h, x, w, torch.full((265,), -100), "bfloat16", scale=2.0)
    assert rec.tolist() == [0.0, 0.0, 0.0, 2.0]
    assert all(bool((y == 0).all()) for y in (losses, dx, dw))
    rec, losses, dx, dw = run_distill(h, x, w, torch.full((265, 3), -1), torch.zeros(265, 3), "bfloat16")
    assert rec.tolist() == [0.0, 0.0, 0.0, 1.0]
    assert all(bool((y == 0).all()) for y in (losses, dx, dw))


@gpu
def test_no_tokens():
    import torch
    x, w, _ = make(1, 40, 600, "bfloat16")
    for tokens in (0, 9):
        h = ar.OutputLoss(tokens, 40, 600)
        rec, _, _, dw = run_ce(h, x[:0], w, torch.zeros(0, dtype=torch.int64), "bfloat16")
        assert rec.tolist() == [0.0, 0.0, 0.0, 1.0] and bool((dw == 0).all())


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_targets_outside_the_vocabulary(dtype):
    import torch
    x, w, g = make(70, 40, 300, dtype, seed=11)
    for wrong in (300, -1, 1 << 40):
        t = targets_of(70, 300, g)
        t[33] = wrong
        h = ar.OutputLoss(70, 40, 300, dtype)
        rec, losses, dx, dw = run_ce(h, x, w, t, dtype)
        assert math.isnan(rec[0].item()) and rec[1].item() == 70 and rec[2].item() == 1.0
        assert losses.isnan().nonzero().tolist() == [[33]]
        assert bool(dx[33].isnan().all()) and not bool(dx[torch.arange(70, device="cuda") != 33].isnan().any())
        assert bool(dw.isnan().all())
    ids, logits = teacher(70, 4, 300, g, "float32")
    h = ar.OutputLoss(70, 40, 300, dtype, top=4)
    for spoil in ("id", "nan", "inf"):
        i2, l2 = ids.clone(), logits.clone()
        if spoil == "id":
            i2[12, 2] = 300
        else:
            l2[12, 2] = float(spoil)
        rec, losses, dx, dw = run_distill(h, x, w, i2, l2, dtype)
        assert losses.isnan().nonzero().tolist() == [[12]] and rec[2].item() == 1.0


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("gain", [20.0, 60.0])
def test_steep_logits(dtype, gain):
    """Logits of tens to hundreds: shares that are 0 or 1 in float32."""
    x, w, g = make(300, 64, 900, dtype, seed=12, gain=gain)
    t = targets_of(300, 900, g, 0.9)
    h = ar.OutputLoss(300, 64, 900, dtype, piece=256)
    Expected(x, w, *one_hot_lists(t), dtype=dtype).check(*run_ce(h, x, w, t, dtype))


@gpu
def test_infinite_logits_say_nonfinite():
    import torch
    x, w, g = make(40, 64, 300, "bfloat16", seed=13)
    x[7] = math.inf
    t = targets_of(40, 300, g)
    h = ar.OutputLoss(40, 64, 300)
    rec, losses, dx, _ = run_ce(h, x, w, t, "bfloat16")
    assert rec[2].item() == 1.0 and not math.isfinite(losses[7].item())
    others = torch.arange(40, device="cuda") != 7
    assert bool(losses[others].isfinite().all()) and bool(dx[others].isfinite().all())


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("d, lead, pad", [(64, 0, 8), (64, 1, 3), (129, 0, 7), (72, 8, 0), (515, 5, 6)])
def test_strided_rows(d, lead, pad, dtype):
    """Rows inside wider ones, off any alignment; what lies between stays."""
    import torch
    n, v = 90, 333
    x, w, g = make(n, d, v, dtype, seed=14)
    t = targets_of(n, v, g, 0.8)

    def inside(y, fill):
        big = torch.full((y.shape[0] * (d + pad) + lead + 64,), fill, dtype=y.dtype, device="cuda")
        view = big[lead:lead + y.shape[0] * (d + pad)].view(y.shape[0], d + pad)[:, :d]
        return big, view
    bx, xv = inside(x, math.nan)
    bw, wv = inside(w, math.nan)
    xv.copy_(x)
    wv.copy_(w)
    bdx, dx = inside(x, 5.0)
    bdw, dw = inside(w, 5.0)
    h = ar.OutputLoss(n, d, v, dtype)
    rec = h.cross_entropy(xv, wv, t.cuda(), grad_hidden=dx, grad_weight=dw)
    h.check()
    Expected(x, w, *one_hot_lists(t), dtype=dtype).check(rec, None, dx, dw)
    for big, view in ((bdx, dx), (bdw, dw)):
        view.fill_(5.0)
        assert bool((big == 5.0).all())


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_fewer_tokens_than_the_handle_is_for(dtype):
    """Stale rows of a larger call before do not show."""
    x, w, g = make(900, 64, 700, dtype, seed=15)
    t = targets_of(900, 700, g)
    h = ar.OutputLoss(900, 64, 700, dtype, top=5, piece=512)
    big = x.clone()
    big[:] = math.nan
    run_ce(h, big, w, t, dtype)
    for n in (1, 255, 600):
        Expected(x[:n], w, *one_hot_lists(t[:n]), dtype=dtype).check(*run_ce(h, x[:n], w, t[:n], dtype))
        ids, logits = teacher(n, 2, 700, g, "float32")
        lists, shares, spread = teacher_lists(ids, logits, 1.0)
        Expected(x[:n], w, lists, shares, dtype=dtype, spread=spread).check(*run_distill(h, x[:n], w, ids, logits, dtype))


@gpu
def test_gradients_against_differences():
    """<gradient, direction> against the definition's central difference along
    it, in 64 bits: off by the gradient's tolerance and h^2 / 6 of the third
    derivative, which for a softmax of logit changes c is below 8 max|c|^3 t^-1."""
    import torch
    n, d, v, t = 40, 64, 500, 2.0
    x, w, g = make(n, d, v, "float32", seed=16)
    ids, logits = teacher(n, 9, v, g, "float32", 0.3)
    h = ar.OutputLoss(n, d, v, "float32", top=9)
    rec, _, dx, dw = run_distill(h, x, w, ids, logits, "float32", temperature=t)
    lists, shares, spread = teacher_lists(ids, logits, t)
    ax, aw = torch.randn(n, d, generator=g).double(), torch.randn(v, d, generator=g).double()
    eps = 1e-5

    def loss(s, by_x, by_w):
        return Expected(x.double().cpu() + s * by_x * ax, w.double().cpu() + s * by_w * aw, lists, shares, t,
                        dtype="float32", spread=spread).loss
    base = Expected(x, w, lists, shares, t, dtype="float32", spread=spread)
    for by_x, by_w, got, a, tol in ((1, 0, dx, ax, base.dx_tol), (0, 1, dw, aw, base.dw_tol)):
        slope = (loss(eps, by_x, by_w) - loss(-eps, by_x, by_w)) / (2 * eps)
        change = float(((by_x * ax) @ w.double().cpu().t() + x.double().cpu() @ (by_w * aw).t()).abs().max())
        room = float((tol * a.abs()).sum()) + U * float((got.double().cpu() * a).abs().sum()) \
            + eps ** 2 / 6 * 8 * change ** 3 / t + 1e-15 * 100 / eps
        assert abs(float((got.double().cpu() * a).sum()) - slope) <= room


@gpu
@pytest.mark.parametrize("n, d, v", [(640, 72, 500), (4, 72, 500)])
def test_in_a_graph_on_its_stream_with_new_inputs(n, d, v):
    import torch
    x, w, g = make(n, d, v, "bfloat16", seed=17)
    t = targets_of(n, v, g, 0.8).cuda()
    h = ar.OutputLoss(n, d, v, top=4, piece=512)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    losses = torch.zeros(n, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec = h.cross_entropy(x, w, t, grad_hidden=dx, grad_weight=dw, losses=losses)
    for seed in (18, 19):
        x2, w2, g2 = make(n, d, v, "bfloat16", seed=seed)
        t2 = targets_of(n, v, g2, 0.3 if seed == 18 else 1.0)
        for a, b in ((x, x2), (w, w2), (t, t2.cuda())):
            a.copy_(b)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
            got = rec.clone(), losses.clone(), dx.clone(), dw.clone()
        side.synchronize()
        h.check()
        Expected(x2, w2, *one_hot_lists(t2)).check(*got)
        eager = run_ce(h, x2, w2, t2, "bfloat16")  # the same bits as the graph's
        assert all(torch.equal(p, q) for p, q in zip(got, eager))


@gpu
def test_weights_packed_in_turn():
    """Float32 rows so long that the workspace holds a part of the weights at a
    time: logits and the gradient of the hidden states go part by part."""
    n, d, v = 40, 65536, 2900
    x, w, g = make(n, d, v, "float32", seed=23)
    t = targets_of(n, v, g, 0.8)
    h = ar.OutputLoss(n, d, v, "float32")
    want = Expected(x, w, *one_hot_lists(t), dtype="float32", on="cuda")
    want.check(*run_ce(h, x, w, t, "float32"))
    want.check(*run_ce(h, x, w, t, "float32", ()))


@gpu
@pytest.mark.parametrize("n", [3, 30])
def test_weights_of_more_than_2_to_the_31_elements(n):
    """Losses, the hidden states' gradient and rows of the weights' from both ends,
    against the definition in pieces of the vocabulary."""
    import torch
    d, v, step = 8192, 270000, 30000
    g = torch.Generator(device="cuda").manual_seed(24)
    x = torch.randn(n, d, generator=g, device="cuda").bfloat16()
    w = torch.empty(v, d, dtype=torch.bfloat16, device="cuda")
    for a in range(0, v, step):
        w[a:a + step] = torch.randn(step, d, generator=g, device="cuda") * (1.3 / math.sqrt(d))
    t = torch.randint(v, (n,), generator=g, device="cuda")
    t[0], t[1] = v - 1, 0
    dw, dx, losses = torch.empty_like(w), torch.empty_like(x), torch.empty(n, device="cuda")
    h = ar.OutputLoss(n, d, v)
    rec = h.cross_entropy(x, w, t, grad_hidden=dx, grad_weight=dw, losses=losses)
    h.check()
    z = torch.cat([x.double() @ w[a:a + step].double().t() for a in range(0, v, step)], 1)
    q = torch.softmax(z, 1)
    want = torch.logsumexp(z, 1) - z.gather(1, t[:, None])[:, 0]
    e = bound_of_sum(d, "bfloat16") * float((x.double().abs().sum(1) * float(w.abs().max())).max())
    dq = 2 * e + 8 * U * (float(z.abs().max()) + 2) + 2 * U * (v + 4) + 16 * U
    assert bool(((losses.double() - want).abs() <= 2 * dq + 4 * U * want).all())
    assert abs(rec[0].item() - float(want.mean())) <= 2 * dq + 8 * U * float(want.mean())
    gz = q.clone()
    gz.scatter_add_(1, t[:, None], torch.full((n, 1), -1.0, dtype=torch.float64, device="cuda"))
    gz /= n
    off = q * dq / n + 2.0 ** -8 * gz.abs() + bound_of_sum(v, "bfloat16") * gz.abs()
    dx_want, room = (torch.zeros(n, d, dtype=torch.float64, device="cuda") for _ in range(2))
    for a in range(0, v, step):
        part = w[a:a + step].double()
        dx_want += gz[:, a:a + step] @ part
        room += off[:, a:a + step] @ part.abs()
    assert bool(((dx.double() - dx_want).abs() <= room * 1.01 + 2.0 ** -8 * dx_want.abs() + 1e-38).all())
    for rows in (slice(0, 300), slice(262000, 262300), slice(v - 300, v)):
        dw_want = gz[:, rows].t() @ x.double()
        room = off[:, rows].t() @ x.double().abs()
        assert bool(((dw[rows].double() - dw_want).abs() <= room * 1.01 + 2.0 ** -8 * dw_want.abs() + 1e-38).all())


@gpu
def test_two_handles_on_two_streams():
    import torch
    cases = []
    for n, d, v, dtype in ((700, 264, 3000, "bfloat16"), (300, 129, 2003, "float32")):
        x, w, g = make(n, d, v, dtype, seed=n)
        t = targets_of(n, v, g, 0.8)
        h = ar.OutputLoss(n, d, v, dtype)
        alone = run_ce(h, x, w, t, dtype)
        cases.append((h, x, w, t.cuda(), alone, torch.cuda.Stream(), [torch.zeros_like(a) for a in (x, w)]))
    torch.cuda.synchronize()
    for _ in range(20):
        for h, x, w, t, _, stream, (dx, dw) in cases:
            h.cross_entropy(x, w, t, grad_hidden=dx, grad_weight=dw, stream=stream)
    torch.cuda.synchronize()
    for h, x, w, t, (rec, _, dx0, dw0), _, (dx, dw) in cases:
        h.check()
        assert torch.equal(h.record, rec) and torch.equal(dx, dx0) and torch.equal(dw, dw0)


@gpu
def test_on_a_stream_that_is_not_current():
    import torch
    x, w, g = make(70, 64, 500, "bfloat16", seed=20)
    t = targets_of(70, 500, g).cuda()
    h, s = ar.OutputLoss(70, 64, 500), torch.cuda.Stream()
    dw, rec = torch.zeros_like(w), torch.zeros(4, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    assert h.cross_entropy(x, w, t, grad_weight=dw, result=rec, stream=s) is rec
    s.synchronize()
    Expected(x, w, *one_hot_lists(t.cpu())).check(rec, None, None, dw)


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n, d, v", [(300, 515, 1003), (40, 1024, 9000), (2000, 128, 300)])
def test_equal_inputs_give_equal_bits(n, d, v, dtype):
    import torch
    x, w, g = make(n, d, v, dtype, seed=21)
    t = targets_of(n, v, g, 0.9)
    h = ar.OutputLoss(n, d, v, dtype)
    first = run_ce(h, x, w, t, dtype)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, run_ce(h, x, w, t, dtype)))


@gpu
def test_refusals():
    import torch
    x, w, g = make(20, 64, 300, "bfloat16")
    t = targets_of(20, 300, g).cuda()
    h = ar.OutputLoss(20, 64, 300, top=4)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)

    def refused(call, **k):
        with pytest.raises((ar.ArError, ValueError)):
            call(**k)
    ce = h.cross_entropy
    refused(ce, hidden=x.float(), weight=w, targets=t)
    refused(ce, hidden=x, weight=w[:299], targets=t)
    refused(ce, hidden=x, weight=w, targets=t[:19])
    refused(ce, hidden=x, weight=w, targets=t.float())
    refused(ce, hidden=x.t().contiguous().t(), weight=w, targets=t)
    refused(ce, hidden=torch.cat([x, x]), weight=w, targets=torch.cat([t, t]))
    refused(ce, hidden=x, weight=w, targets=t, scale=0.0)
    refused(ce, hidden=x, weight=w, targets=t, scale=math.nan)
    refused(ce, hidden=x, weight=w, targets=t, grad_hidden=x)
    refused(ce, hidden=x, weight=w, targets=t, grad_weight=w)
    refused(ce, hidden=x, weight=w, targets=t, grad_hidden=w[:20])
    refused(ce, hidden=x, weight=w, targets=t, grad_hidden=dx[:1].expand(20, 64))
    refused(ce, hidden=x, weight=w, targets=t, grad_weight=dw.half())
    refused(ce, hidden=x, weight=w, targets=t, losses=torch.zeros(19, device="cuda"))
    refused(ce, hidden=x, weight=w, targets=t, result=torch.zeros(3, device="cuda"))
    ids, logits = torch.zeros(20, 4, dtype=torch.int64, device="cuda"), torch.zeros(20, 4, device="cuda")
    for k in (dict(temperature=0.0), dict(temperature=math.inf), dict(temperature=1e30),
              dict(temperature=1e-30), dict(ids=ids[:, :3]), dict(logits=logits.half()),
              dict(ids=torch.zeros(20, 5, dtype=torch.int64, device="cuda"), logits=torch.zeros(20, 5, device="cuda")),
              dict(ids=ids[:, :0], logits=logits[:, :0])):
        refused(h.distill, **{**dict(hidden=x, weight=w, ids=ids, logits=logits), **k})
    small = ar.OutputLoss(20, 64, 300, grads=False)
    refused(small.cross_entropy, hidden=x, weight=w, targets=t, grad_weight=dw)
    L, a = ar.lib(), h._args(x, w, "mean", 1.0, dx, dw, False, None, None)
    s = torch.cuda.current_stream().cuda_stream
    host = torch.zeros(20, dtype=torch.int64)
    assert L.ar_output_cross_entropy(h._h, ctypes.byref(a), host.data_ptr(), 8, -100, s) == 1
    assert L.ar_output_cross_entropy(h._h, ctypes.byref(a), t.data_ptr(), 2, -100, s) == 1
    assert L.ar_output_cross_entropy(h._h, ctypes.byref(a), t.data_ptr() + 1, 8, -100, s) == 1
    a.weight_stride = 1 << 30
    assert L.ar_output_cross_entropy(h._h, ctypes.byref(a), t.data_ptr(), 8, -100, s) == 1
    a.weight_stride = 63
    assert L.ar_output_cross_entropy(h._h, ctypes.byref(a), t.data_ptr(), 8, -100, s) == 1
    torch.cuda.synchronize()
    Expected(x, w, *one_hot_lists(t.cpu())).check(*run_ce(h, x, w, t.cpu(), "bfloat16"))  # goes on after them


@gpu
def test_backward_over_a_gradient_from_before_the_call_is_an_error():
    import torch
    x, w, g = make(20, 64, 300, "float32")
    h = ar.OutputLoss(20, 64, 300, "float32")
    dx = torch.zeros_like(x)
    y = torch.ones_like(x).requires_grad_()
    z = (y * dx).sum()
    h.cross_entropy(x, w, targets_of(20, 300, g).cuda(), grad_hidden=dx)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()


@gpu
def test_loss_then_norm_then_update():
    """The operators as a step uses them: gradients of two losses added, their
    norm, the update; a wrong target skips the update."""
    import torch
    n, d, v = 120, 64, 700
    x, w, g = make(n, d, v, "bfloat16", seed=22)
    t = targets_of(n, v, g, 0.8)
    ids, logits = teacher(n, 6, v, g, "float32")
    master = w.float()
    dw = torch.zeros(v, d, device="cuda")
    h = ar.OutputLoss(n, d, v, top=6)
    grads = ar.Grads([dw])
    opt = ar.AdamW([master], [dw], [torch.zeros_like(dw)], [torch.zeros_like(dw)], copies=[w])
    before = w.clone()
    h.cross_entropy(x, w, t.cuda(), scale=0.5, grad_weight=dw)
    h.distill(x, w, ids.cuda(), logits.cuda(), scale=0.5, grad_weight=dw, accumulate=True)
    record = grads.norm(max_norm=1.0)
    opt.step(1, lr=1e-2, clip=record)
    lists, shares, spread = teacher_lists(ids, logits, 1.0)
    ce = Expected(x, before, *one_hot_lists(t), scale=0.5)
    kd = Expected(x, before, lists, shares, scale=0.5, spread=spread)
    want, room = ce.dw + kd.dw, ce.dw_tol + kd.dw_tol
    assert bool(((dw.double().cpu() - want).abs() <= room * (1 + 4 * U) + 4 * U * (ce.dw.abs() + kd.dw.abs())).all())
    norm = float(dw.double().norm())
    assert record[0].item() == pytest.approx(norm, rel=10 * U)
    assert not torch.equal(w, before) and torch.equal(w, master.bfloat16())
    t[5] = v
    h.cross_entropy(x, w, t.cuda(), grad_weight=dw)
    after = master.clone()
    opt.step(2, lr=1e-2, clip=grads.norm(max_norm=1.0))
    assert torch.equal(master, after)


@gpu
@pytest.mark.parametrize("teacher_k", [0, 6])
def test_sharded_step_of_an_output_layer(teacher_k):
    """examples/zero_step.py with ar.OutputLoss: every rank's float32 gradient,
    the update that follows from them, and the same bits from its graph."""
    import sys
    import torch
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import zero_step
    P, n, d, v = 3, 70, 40, 331
    eager, graphed = (zero_step.OutputLayerStep(P, n, d, v, teacher_k, weight_decay=0.01) for _ in range(2))
    graph = graphed.capture()
    for _ in range(3):
        before = [w.clone().view(v, d) for w in eager.weights]
        eager.backward()
        for r in range(P):
            if teacher_k:
                lists, shares, spread = teacher_lists(eager.ids[r].cpu(), eager.top[r].cpu(), 1.0)
                want = Expected(eager.states[r], before[r], lists, shares, spread=spread)
            else:
                want = Expected(eager.states[r], before[r], *one_hot_lists(eager.next[r].cpu()))
            want.check(eager.records[r], None, None, eager.grads[r].view(v, d))
        mean = sum(g.double() for g in eager.grads) / P
        record = eager.step()
        assert record[0].item() == pytest.approx(float(mean.norm()), rel=(10 + 2 * P) * U)
        assert all(torch.equal(eager.weights[0], w) for w in eager.weights)
        assert not torch.equal(eager.weights[0].view(v, d), before[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager.records, graphed.records)
        assert all(torch.equal(p, q) for p, q in zip(eager.weights + eager.master, graphed.weights + graphed.master))
    eager.loss.check()
    graphed.loss.check()


@gpu
def test_closing_twice_and_dropping_during_a_capture():
    import torch
    x, w, g = make(20, 64, 300, "bfloat16")
    t = targets_of(20, 300, g).cuda()
    h, other = ar.OutputLoss(20, 64, 300), ar.OutputLoss(20, 64, 300)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec = h.cross_entropy(x, w, t)
        del other
    graph.replay()
    torch.cuda.synchronize()
    assert rec[1].item() == 20.0
    h.close()
    h.close()
    with pytest.raises(ar.ArError):
        h.cross_entropy(x, w, t)
