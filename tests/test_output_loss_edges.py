"""The output layer's losses where what is read, asked for or summed could make
them go wrong: NaN and infinities in the weights and hidden states, rows that are
far apart, float32 gradients of bf16 inputs, sums over a million products, odd
views of weights, parts of them in turn, elements behind 2^31.

Tolerances as derived in test_output_loss.py, with the products of a logit that
are not zero in the place of all of them (adding a zero rounds nothing), and on
the gradient of a logit the rounding that the call makes: to bf16, or none
beyond float32's."""

import ctypes
import math
import os
import subprocess

import pytest

import collective_reduction_gb300 as ar
from test_output_loss import (Expected, U, bound_of_sum, half_step, make, run_ce, run_distill, targets_of, tdt, teacher,
                              teacher_lists)

gpu = pytest.mark.gpu
HALF = 2.0 ** -8  # of a step of bf16, relative


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    return ensure_built()


class Tight:
    """Softmax cross entropy in 64 bits and how far a call may be off it.  `terms`:
    products of a logit that are not zero; `half`: half a step, relative, of the
    logits' gradients; `out`: entry whose logit is -infinity."""

    def __init__(self, x, w, targets, dtype, terms=None, half=U, ignore=-100, reduction="mean", scale=1.0, out=None):
        import torch
        x, w, t = x.double(), w.double(), targets.cuda()
        n, v = x.shape[0], w.shape[0]
        counted = t != ignore
        mask = counted.double()[:, None]
        x = torch.where(counted[:, None], x, 0.0)
        self.counted = int(counted.sum())
        self.factor = scale / max(1, self.counted) if reduction == "mean" else scale
        z = x @ w.t()
        if out is not None:
            z[:, out] = -math.inf
        at = torch.where(counted, t, 0).long()[:, None]
        p = torch.zeros_like(z).scatter_(1, at, 1.0)
        lse = torch.logsumexp(z, 1, keepdim=True)
        self.losses = ((lse - z.gather(1, at)) * mask)[:, 0]
        self.loss = float(self.losses.sum()) * self.factor
        q = (z - lse).exp()
        g = self.factor * (q - p) * mask
        if out is None:
            e = bound_of_sum(terms or x.shape[1], dtype) * (x.abs() @ w.abs().t()).amax(1, keepdim=True)
            big = z.abs().amax(1, keepdim=True)
        else:
            keep = torch.arange(v, device="cuda") != out
            e = bound_of_sum(terms or x.shape[1], dtype) * (x.abs() @ w[keep].abs().t()).amax(1, keepdim=True)
            big = z[:, keep].abs().amax(1, keepdim=True)
        d = 2 * e + 8 * U * (big + 2) + 2 * U * (v + 4) + 16 * U
        self.losses_tol = (2 * d * mask)[:, 0] + 4 * U * self.losses
        self.loss_tol = float(self.losses_tol.sum()) * self.factor + 4 * U * abs(self.loss)
        if out is not None:
            return
        g_tol = self.factor * (q * d + p * 4 * U) * mask + (half + 4 * U) * g.abs()
        kind = "float32" if half == U else dtype  # the planes' products are as many as float32's at most
        self.dx, self.dw = g @ w, g.t() @ x
        self.dx_tol = g_tol @ w.abs() + bound_of_sum(v, kind) * (g.abs() @ w.abs())
        self.dw_tol = g_tol.t() @ x.abs() + bound_of_sum(n, kind) * (g.abs().t() @ x.abs())

    def check(self, record, losses=None, dx=None, dw=None, old=0.0, telling=0.5):
        """`telling`: the part of the gradients' elements at least that results of
        zeros would fail at."""
        loss, counted, nonfinite, factor = record.tolist()
        assert counted == self.counted and nonfinite == 0.0 and factor == pytest.approx(self.factor, rel=2 * U)
        assert abs(loss - self.loss) <= self.loss_tol < abs(self.loss)
        if losses is not None:
            assert bool(((losses.double() - self.losses).abs() <= self.losses_tol).all())
        for got, want, tol in ((dx, self.dx, self.dx_tol), (dw, self.dw, self.dw_tol)):
            if got is None:
                continue
            want = want + old
            half = half_step(str(got.dtype).replace("torch.", ""))
            room = tol + (half + 2 * U) * (want.abs() + tol) + 1e-38
            assert float((want.abs() > room)[want != 0].double().mean()) >= telling
            off = (got.double() - want).abs()
            assert bool((off <= room).all()), float((off / room).max())


def sparse_states(n, d, cols, g, dtype):
    """Hidden states that are zero but in `cols` columns, spread from the first to the last."""
    import torch
    at = torch.linspace(0, d - 1, cols).round().long().cuda()
    x = torch.zeros(n, d, dtype=tdt(dtype), device="cuda")
    x[:, at] = torch.randn(n, cols, generator=g, device="cuda").to(x.dtype)
    return x, at


# ------------------------------------------------- what is not a number

def avoid(t, entry, v):
    t = t.clone()
    t[t == entry] = (entry + 1) % v
    return t


def columns_of(v):
    return sorted({c for c in (0, 5, 31, 32, 63, 64, 127, 128, 255, 256, v - 1) if c < v})


FEW_AND_TILES = [("bfloat16", 1, 64, 65), ("bfloat16", 2, 33, 129), ("bfloat16", 3, 64, 257), ("bfloat16", 8, 40, 300),
                 ("float32", 1, 33, 129), ("float32", 8, 64, 257), ("float32", 12, 1100, 2003),
                 ("bfloat16", 40, 64, 129), ("bfloat16", 300, 40, 257), ("bfloat16", 40, 33, 65), ("float32", 40, 64, 129),
                 ("float32", 300, 33, 257), ("float32", 300, 40, 300)]


@gpu
@pytest.mark.parametrize("dtype, n, d, v", FEW_AND_TILES)
@pytest.mark.parametrize("grads", [(), ("hidden", "weight")])
def test_a_nan_weight_makes_every_loss_nan(dtype, n, d, v, grads):
    """Also where it is the only entry of a part of the vocabulary, or its first."""
    x, w, g = make(n, d, v, dtype, seed=n + v)
    t0 = targets_of(n, v, g, 0.8)
    t0[0] = 1
    h = ar.OutputLoss(n, d, v, dtype, top=2)
    ids, logits = teacher(n, 2, v, g, "float32")
    for c in columns_of(v):
        w2, t = w.clone(), avoid(t0, c, v)
        w2[c, d // 2] = math.nan
        rec, losses, dx, dw = run_ce(h, x, w2, t, dtype, grads)
        counts = (t != -100).cuda()
        assert math.isnan(rec[0].item()) and rec[1].item() == int(counts.sum()) and rec[2].item() == 1.0, c
        assert bool(losses[counts].isnan().all()) and bool((losses[~counts] == 0).all()), c
        if grads:
            assert bool(dw.isnan().all()) and bool(dx[counts].isnan().all()) and bool((dx[~counts] == 0).all()), c
        rec, losses, _, _ = run_distill(h, x, w2, avoid(ids, c, v), logits, dtype)
        assert rec[2].item() == 1.0 and bool(losses.isnan().all()), c


@gpu
@pytest.mark.parametrize("dtype, n, d, v", FEW_AND_TILES)
def test_an_infinite_weight(dtype, n, d, v):
    """A logit of -infinity adds nothing, one of +infinity leaves no finite loss.  The
    tensor cores' float32 products of an infinity may be NaN instead: never a
    finite loss that is wrong."""
    import torch
    x, w, g = make(n, d, v, dtype, seed=n + v)
    x[:, 0] = torch.where(torch.rand(n, generator=g).cuda() < 0.5, x[:, 0].abs() + 0.1, -x[:, 0].abs() - 0.1)
    t0 = targets_of(n, v, g)
    planes = dtype == "float32" and n > 24
    h = ar.OutputLoss(n, d, v, dtype)
    for c in columns_of(v):
        t = avoid(t0, c, v)
        want = Tight(x, w, t, dtype, out=c)
        for sign in (1.0, -1.0):
            w2 = w.clone()
            w2[c, 0] = sign * math.inf
            up = x[:, 0] * sign > 0
            rec, losses, _, _ = run_ce(h, x, w2, t, dtype, ())
            assert not bool(losses[up].isfinite().any()) and rec[2].item() == float(bool((~losses.isfinite()).any())), c
            off = (losses.double() - want.losses).abs()
            right = off <= want.losses_tol
            assert bool((right | up | (planes & ~losses.isfinite())).all()), c


@gpu
@pytest.mark.parametrize("dtype, n", [("bfloat16", 3), ("bfloat16", 40), ("float32", 3), ("float32", 40)])
def test_a_nan_hidden_state_is_its_tokens_alone(dtype, n):
    import torch
    x, w, g = make(n, 64, 257, dtype, seed=n)
    t = targets_of(n, 257, g)
    x[1, 5] = math.nan
    rec, losses, dx, dw = run_ce(ar.OutputLoss(n, 64, 257, dtype), x, w, t, dtype)
    others = torch.arange(n, device="cuda") != 1
    assert rec[2].item() == 1.0 and math.isnan(losses[1].item()) and bool(losses[others].isfinite().all())
    assert bool(dx[1].isnan().all()) and bool(dx[others].isfinite().all()) and bool(dw.isnan().all())


# ------------------------------------------------- what counts

@gpu
@pytest.mark.parametrize("n", [5, 300])
@pytest.mark.parametrize("ignore, size", [(7, 4), (7, 8), (-1, 4), (0, 8), (1 << 40, 8)])
def test_another_ignore_index(n, ignore, size):
    import torch
    x, w, g = make(n, 64, 300, "bfloat16", seed=n)
    t = targets_of(n, 300, g)
    t[::3] = ignore
    h = ar.OutputLoss(n, 64, 300)
    rec, losses, dx, dw = run_ce(h, x, w, t if size == 8 else t.int(), "bfloat16", ignore_index=ignore)
    Tight(x, w, t, "bfloat16", half=HALF, ignore=ignore).check(rec, losses, dx, dw)
    assert bool((losses[(t == ignore).cuda()] == 0).all())
    if ignore >= 0:  # and -100 is a target like others then: outside the vocabulary
        t[1] = -100
        rec, losses, _, _ = run_ce(h, x, w, t if size == 8 else t.int(), "bfloat16", ignore_index=ignore)
        assert rec[2].item() == 1.0 and math.isnan(losses[1].item())


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n, d, v", [(1, 64, 300), (7, 129, 2003), (12, 1100, 2003), (40, 33, 65), (513, 96, 2003),
                                     (2000, 40, 257)])
@pytest.mark.parametrize("keep", [1.0, 0.5])
def test_handles_for_losses_alone(n, d, v, dtype, keep):
    """Also for fewer tokens than the handle's, and with a teacher's lists."""
    import torch
    x, w, g = make(n, d, v, dtype, seed=n + d)
    t = targets_of(n, v, g, keep)
    t[0] = 1
    h = ar.OutputLoss(n + 300, d, v, dtype, top=5, grads=False)
    assert h.info()["pieces"] == 1
    Tight(x, w, t, dtype).check(*run_ce(h, x, w, t, dtype, ()))
    ids, logits = teacher(n, 5, v, g, dtype, 1.0 - keep, twice=True)
    losses = torch.full((n,), 7.0, device="cuda")
    rec = h.distill(x, w, ids.cuda(), logits.cuda(), temperature=2.0, losses=losses)
    h.check()
    lists, shares, spread = teacher_lists(ids, logits, 2.0)
    Expected(x, w, lists, shares, 2.0, dtype=dtype, spread=spread).check(rec, losses)


# ------------------------------------------------- rows that are far apart

FAR = [(4, 1 << 22, 1 << 40), (2, 1 << 23, 1 << 40), (2, 1 << 24, 1 << 39), (8, 1 << 21, 1 << 40), (4, 3, (1 << 63) - 1),
       (2, 2, (1 << 64) - 1)]


def test_bytes_of_rows_that_are_far_apart_do_not_wrap(tmp_path):
    """Sizes whose rows times stride times element are a multiple of 2^64, and
    ordinary ones, as the checks of a call compute them, on the host alone."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cases = [(r + 1, 8, s, e) for e, r, s in FAR] + [(0, 8, 8, 2), (5, 0, 8, 2), (1, 8, 1 << 60, 4), (1, 1 << 62, 1 << 62, 4),
                                                     (3, 5, 7, 2), (1 << 24, 1 << 16, 1 << 16, 4), (1 << 21, 1, 1 << 39, 4)]
    lines = "\n".join(f'    std::printf("%llu\\n", (unsigned long long)ar::matrix_bytes({r}ull, {w}ull, {s}ull, {e}ull));'
                      for r, w, s, e in cases)
    source = tmp_path / "bytes.cpp"
    source.write_text(f'#include <cstdio>\n#include "bufcheck.hpp"\nint main() {{\n{lines}\n}}\n')
    program = tmp_path / "bytes"
    subprocess.run(["g++", "-std=c++17", "-I" + os.path.join(root, "include"), "-I/usr/local/cuda/include",
                    "-I" + os.path.join(root, "collective_reduction_gb300", "csrc"), str(source), "-o", str(program)],
                   check=True)
    got = subprocess.run([str(program)], check=True, capture_output=True, text=True).stdout.split()
    for (r, w, s, e), b in zip(cases, got):
        exact = ((r - 1) * s + w) * e if r and w else 0
        assert int(b) == (exact if exact < 1 << 62 else (1 << 64) - 1), (r, w, s, e)


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_weights_whose_rows_are_far_apart_are_refused(dtype):
    """By the host, before any launch."""
    import torch
    v = (1 << (23 if dtype == "bfloat16" else 22)) + 1
    x, w = (torch.zeros(8 * k, dtype=getattr(torch, dtype), device="cuda") for k in (1, 64))
    targets = torch.zeros(1, dtype=torch.int64, device="cuda")
    h = ar.OutputLoss(1, 8, v, dtype, grads=False)
    a = ar.OutputLossArgs()
    a.tokens, a.hidden, a.hidden_stride, a.scale, a.result = 1, x.data_ptr(), 8, 1.0, h.record.data_ptr()
    a.weight = w.data_ptr()
    for stride in (1 << 40, 1 << 39, (1 << 64) - 1):
        a.weight_stride = stride
        assert ar.lib().ar_output_cross_entropy(h._h, ctypes.byref(a), targets.data_ptr(), 8, -100, None) == 1
    h.check()
    assert bool((h.record == 0).all())


# ------------------------------------------------- float32 gradients of bf16 inputs

@gpu
@pytest.mark.parametrize("n, d, v, piece", [(20, 64, 300, 0), (300, 515, 1003, 0), (900, 72, 700, 0), (900, 72, 700, 256),
                                            (2400, 136, 257, 256)])
@pytest.mark.parametrize("grads", [("hidden", "weight"), ("hidden",), ("weight",)])
def test_float32_gradients_of_bf16_inputs_are_of_float32_logit_gradients(n, d, v, piece, grads):
    import torch
    x, w, g = make(n, d, v, "bfloat16", seed=n)
    t = targets_of(n, v, g, 0.8)
    h = ar.OutputLoss(n, d, v, piece=piece)
    want = Tight(x, w, t, "bfloat16")
    rec, losses, dx, dw = run_ce(h, x, w, t, "bfloat16", grads, "float32")
    want.check(rec, losses, dx, dw)
    old = {k: 0.25 for k in grads}
    more = {"grad_" + k: torch.full(y.shape, old[k], device="cuda") for k, y in (("hidden", x), ("weight", w)) if k in grads}
    rec = h.cross_entropy(x, w, t.cuda(), accumulate=True, **more)
    h.check()
    want.check(rec, None, more.get("grad_hidden"), more.get("grad_weight"), old=0.25)


@gpu
@pytest.mark.parametrize("wide", ["hidden", "weight"])
@pytest.mark.parametrize("piece", [0, 256])
def test_one_gradient_in_float32_and_one_in_bf16(wide, piece):
    import torch
    n, d, v = 900, 72, 700
    x, w, g = make(n, d, v, "bfloat16", seed=3)
    t = targets_of(n, v, g, 0.8)
    h = ar.OutputLoss(n, d, v, piece=piece)
    dx = torch.full((n, d), 7.0, device="cuda", dtype=torch.float32 if wide == "hidden" else torch.bfloat16)
    dw = torch.full((v, d), 7.0, device="cuda", dtype=torch.float32 if wide == "weight" else torch.bfloat16)
    losses = torch.full((n,), 7.0, device="cuda")
    rec = h.cross_entropy(x, w, t.cuda(), grad_hidden=dx, grad_weight=dw, losses=losses).clone()
    h.check()
    exact, rounded = Tight(x, w, t, "bfloat16"), Tight(x, w, t, "bfloat16", half=HALF)
    exact.check(rec, losses, dx if wide == "hidden" else None, dw if wide == "weight" else None)
    rounded.check(rec, losses, dx if wide != "hidden" else None, dw if wide != "weight" else None)


@gpu
@pytest.mark.parametrize("n", [1, 2, 5, 8])
@pytest.mark.parametrize("d, v", [(64, 300), (129, 517), (1024, 600), (8192, 520), (16384, 700), (65536, 560)])
def test_a_few_tokens_gradients_are_rounded_once(n, d, v):
    """Whatever the weights' size: 0.04 to 73 MB."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(n + d)
    x, _ = sparse_states(n, d, 16, g, "bfloat16")
    w = (0.4 * torch.randn(v, d, generator=g, device="cuda")).bfloat16()
    t = torch.randint(v, (n,), generator=g, device="cuda")
    rec, losses, dx, dw = run_ce(ar.OutputLoss(n, d, v), x, w, t, "bfloat16")
    Tight(x, w, t, "bfloat16", terms=16).check(rec, losses, dx, dw)


@gpu
@pytest.mark.parametrize("n, d, v, k", [(6, 1024, 3000, 5), (300, 72, 2003, 33), (900, 40, 300, 300)])
def test_float32_gradients_of_a_distillation(n, d, v, k):
    """Entries of one id add up, some are absent; twice the same bits, also from a graph
    that is given new inputs."""
    import torch
    x, w, g = make(n, d, v, "bfloat16", seed=k)
    h = ar.OutputLoss(n, d, v, top=k, piece=512)
    dx, dw, losses = (torch.zeros(s, device="cuda") for s in ((n, d), (v, d), (n,)))
    ids, logits = (y.cuda() for y in teacher(n, k, v, g, "float32", 0.3, twice=True))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec = h.distill(x, w, ids, logits, temperature=2.0, grad_hidden=dx, grad_weight=dw, losses=losses)
    for seed in (41, 42):
        ids2, logits2 = teacher(n, k, v, g.manual_seed(seed), "float32", 0.3, twice=True)
        ids.copy_(ids2)
        logits.copy_(logits2)
        graph.replay()
        h.check()
        lists, shares, spread = teacher_lists(ids2, logits2, 2.0)
        want = Expected(x, w, lists, shares, 2.0, dtype="float32", spread=spread)
        want.check(rec, losses, dx, dw)
        assert bool((want.dw.abs() > want.dw_tol)[want.dw != 0].double().mean() > 0.5)
        first = [y.clone() for y in (rec, losses, dx, dw)]
        h.distill(x, w, ids, logits, temperature=2.0, grad_hidden=dx, grad_weight=dw, losses=losses)
        assert all(torch.equal(a, b) for a, b in zip(first, (rec, losses, dx, dw)))


@gpu
@pytest.mark.parametrize("n", [6, 70, 700])
def test_float32_gradients_of_a_target_outside_the_vocabulary(n):
    import torch
    x, w, g = make(n, 1024, 3001, "bfloat16", seed=n)
    t = targets_of(n, 3001, g)
    t[4] = 3001
    rec, losses, dx, dw = run_ce(ar.OutputLoss(n, 1024, 3001, piece=256), x, w, t, "bfloat16", gtype="float32")
    others = torch.arange(n, device="cuda") != 4
    assert rec[2].item() == 1.0 and losses.isnan().nonzero().tolist() == [[4]]
    assert bool(dx[4].isnan().all()) and bool(dx[others].isfinite().all()) and bool(dw.isnan().all())


@gpu
def test_float32_and_bf16_gradients_on_two_streams_are_as_alone():
    import torch
    n, d, v = 700, 264, 3000
    x, w, g = make(n, d, v, "bfloat16", seed=6)
    t = targets_of(n, v, g, 0.8)
    cases = []
    for gtype in ("float32", "bfloat16"):
        h = ar.OutputLoss(n, d, v)
        alone = run_ce(h, x, w, t, "bfloat16", gtype=gtype)
        cases.append((h, alone, torch.cuda.Stream(), [torch.zeros_like(a) for a in alone[2:]]))
    t = t.cuda()
    torch.cuda.synchronize()
    for _ in range(20):
        for h, _, stream, (dx, dw) in cases:
            h.cross_entropy(x, w, t, grad_hidden=dx, grad_weight=dw, stream=stream)
    torch.cuda.synchronize()
    for h, (rec, _, dx0, dw0), _, (dx, dw) in cases:
        h.check()
        assert torch.equal(h.record, rec) and torch.equal(dx, dx0) and torch.equal(dw, dw0)


# ------------------------------------------------- long sums

def rows_near_two(rows, width, seed):
    """Random bf16 in [1.8, 2)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    y = torch.empty(rows, width, dtype=torch.bfloat16, device="cuda")
    for part in y.split(1 << 18):
        part.copy_(1.8 + 0.19 * torch.rand(part.shape, generator=g, device="cuda"))
    return y


# 65536 additions in the tensor cores, each cut off below 2^-23, are 0.13% of such sums: 0.6 of half
# a step of bf16 at values just below a power of two.  Runs of at most 256 blocks of four additions:
LONG_SUM = 256 * 4 * 2 * U + (1 << 20) // (256 * 64) * U + 16 * U


@gpu
def test_bf16_gradient_of_weights_over_a_million_tokens():
    """Terms of one sign: every logit is 0, so a row that is no target is the sum of all
    hidden states / 1024.  76 tiles: nothing is gained by splitting the sums."""
    import torch
    n, d, v = 1 << 20, 4864, 1024
    x = rows_near_two(n, d, 31)
    w, dw = (torch.zeros(v, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    h = ar.OutputLoss(n, d, v)
    rec = h.cross_entropy(x, w, torch.zeros(n, dtype=torch.int32, device="cuda"), reduction="sum", grad_weight=dw)
    h.check()
    want = sum(part.double().sum(0) for part in x.split(1 << 18)) / v
    assert 1024.0 < float(want.min()) and float(want.max()) < 2048.0
    assert bool(((dw[1:].double() - want).abs() <= 4.0 + LONG_SUM * want).all())  # half a step
    assert rec[0].item() == pytest.approx(n * math.log(v), rel=1e-6)


@gpu
def test_bf16_gradient_of_hidden_states_over_a_million_entries():
    """Hidden states of 0 and a target's row of 0: the mean of the other rows."""
    import torch
    n, d, v = 1024, 4864, 1 << 20
    w = rows_near_two(v, d, 32)
    w[7] = 0
    x, dx = (torch.zeros(n, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    h = ar.OutputLoss(n, d, v)
    rec = h.cross_entropy(x, w, torch.full((n,), 7, device="cuda"), reduction="sum", scale=16.0, grad_hidden=dx)
    h.check()
    want = 16.0 * sum(part.double().sum(0) for part in w.split(1 << 18)) / v
    assert 16.0 < float(want.min()) and float(want.max()) < 32.0
    assert bool(((dx.double() - want).abs() <= 0.0625 + LONG_SUM * want).all())
    assert rec[0].item() == pytest.approx(16 * n * math.log(v), rel=1e-6)


# ------------------------------------------------- memory

def test_workspace_is_that_of_what_calls_use():
    """Handles for a few tokens pack no weights, others of bf16 rows of whole 16 bytes
    256 MB of them at most; the weights' gradient takes a sum of its own only where
    bf16 is asked of runs of pieces."""
    mb = 1 << 20
    for dtype in ("bfloat16", "float32"):
        few = ar.output_loss_layout(8, 4096, 128000, dtype, grads=False)["workspace_bytes"]
        assert few < 256 * 4096 * 6 * 2 + 16 * mb  # a tile of states and of weights
    scored = ar.output_loss_layout(16384, 4096, 128000, grads=False)["workspace_bytes"]
    assert scored < 2 * 16384 * 4096 + 256 * mb + 8 * 16384 * 1000 + 8 * mb  # states, odd views, statistics
    assert ar.output_loss_layout(37, 129, 2003, "float32")["workspace_bytes"] < 32 * mb
    bf16, f32 = (ar.output_loss_layout(4096, 1024, 50001, t, piece=256)["workspace_bytes"] for t in ("bfloat16", "float32"))
    wide = 50176  # logits of 256 tokens, gradients of 1024, hidden states, weights (packed: all), parts, the sum
    assert bf16 < wide * (4 * 256 + 2 * 1024) + 4096 * 1024 * 2 + 256 * mb + 160 * mb + wide * 1024 * 4
    assert f32 < wide * (4 * 256 + 6 * 1024) + 4096 * 1024 * 6 + wide * 1024 * 6 + 160 * mb


@gpu
@pytest.mark.parametrize("gtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n", [3, 300])
def test_odd_views_of_weights_are_packed_in_turn(n, gtype):
    """328 MB of bf16 rows whose pitch is no multiple of 16 bytes."""
    import torch
    d, v = 2048, 80000
    g = torch.Generator(device="cuda").manual_seed(35)
    x, _ = sparse_states(n, d, 24, g, "bfloat16")
    w = (0.3 * torch.randn(v, d, generator=g, device="cuda")).bfloat16()
    odd = torch.full((v, d + 1), math.nan, dtype=torch.bfloat16, device="cuda")[:, 1:]
    odd.copy_(w)
    t = torch.randint(v, (n,), generator=g, device="cuda")
    part = (1 << 28) // (2 * d) // 256 * 256  # entries at a time
    t[:3] = torch.tensor([part - 1, part, v - 1], device="cuda")
    h = ar.OutputLoss(n, d, v)
    assert 0 < part < v
    half = U if n <= 8 or gtype == "float32" else HALF
    want = Tight(x, w, t, "bfloat16", terms=24, half=half)
    want.check(*run_ce(h, x, odd, t, "bfloat16", gtype=gtype), telling=0.2)
    want.check(*run_ce(h, x, odd, t, "bfloat16", (), gtype))


@gpu
@pytest.mark.parametrize("n, keep", [(12, 1.0), (21, 0.6), (24, 1.0), (25, 1.0), (40, 1.0), (40, 0.6)])
def test_weights_packed_in_turn_element_by_element(n, keep):
    """Float32 rows of 65536: a part of 2560 entries is packed at a time, or up to 24
    tokens go in groups that read them as they are.  The states' 24 values a row
    leave logits that are off by 1e-4 at most."""
    import torch
    d, v = 65536, 2900
    g = torch.Generator(device="cuda").manual_seed(33)
    x, at = sparse_states(n, d, 24, g, "float32")
    w = torch.randn(v, d, generator=g, device="cuda") * 0.4
    t = torch.randint(v, (n,), generator=g, device="cuda")
    t[torch.rand(n, generator=g, device="cuda") >= keep] = -100
    t[:4] = torch.tensor([0, 2559, 2560, v - 1], device="cuda")
    h = ar.OutputLoss(n, d, v, "float32")
    want = Tight(x, w, t, "float32", terms=24)
    rec, losses, dx, dw = run_ce(h, x, w, t, "float32")
    want.check(rec, losses, dx, dw)
    want.check(*run_ce(h, x, w, t, "float32", ()))
    dx0 = torch.ones_like(dx)
    want.check(h.cross_entropy(x, w, t, grad_hidden=dx0, accumulate=True), None, dx0, old=1.0)


@gpu
@pytest.mark.parametrize("n", [3, 30])
def test_rows_around_element_2_to_the_31(n):
    """Losses, the hidden states' gradient and every row of the weights', with targets
    on both sides of the boundary and at both ends."""
    import torch
    d, v, step = 8192, 270000, 30000
    edge = (1 << 31) // d
    g = torch.Generator(device="cuda").manual_seed(34)
    x, at = sparse_states(n, d, 16, g, "bfloat16")
    w = torch.empty(v, d, dtype=torch.bfloat16, device="cuda")
    for a in range(0, v, step):
        w[a:a + step] = torch.randn(step, d, generator=g, device="cuda")
    t = torch.randint(v, (n,), generator=g, device="cuda")
    t[:3] = torch.tensor([edge - 1, edge, v - 1], device="cuda")
    if n > 3:
        t[3] = 0
    dw, dx, losses = torch.full_like(w, 7.0), torch.empty_like(x), torch.empty(n, device="cuda")
    h = ar.OutputLoss(n, d, v)
    rec = h.cross_entropy(x, w, t, reduction="sum", grad_hidden=dx, grad_weight=dw, losses=losses)
    h.check()
    # the definition with the columns that are not zero, but for the states' gradient
    half = U if n <= 8 else HALF
    small = Tight(x[:, at], w[:, at], t, "bfloat16", half=half, reduction="sum")
    small.check(rec, losses, None, dw[:, at])
    rest = torch.ones(d, dtype=torch.bool, device="cuda")
    rest[at] = False
    z = x[:, at].double() @ w[:, at].double().t()
    q = torch.softmax(z, 1)
    gz = q.scatter_add(1, t[:, None], torch.full((n, 1), -1.0, dtype=torch.float64, device="cuda"))
    e = bound_of_sum(16, "bfloat16") * float((x[:, at].double().abs() @ w[:, at].double().abs().t()).max())
    dq = 2 * e + 8 * U * (float(z.abs().max()) + 2) + 2 * U * (v + 4) + 16 * U
    off = q * dq + gz.abs() * (half + bound_of_sum(v, "bfloat16") + 4 * U)
    want, room = (torch.zeros(n, d, dtype=torch.float64, device="cuda") for _ in range(2))
    for a in range(0, v, step):
        assert bool((dw[a:a + step][:, rest] == 0).all())
        part = w[a:a + step].double()
        want += gz[:, a:a + step] @ part
        room += off[:, a:a + step] @ part.abs()
    room += HALF * (want.abs() + room) + 1e-38
    assert float((want.abs() > room).double().mean()) > 0.5
    assert bool(((dx.double() - want).abs() <= room).all())
