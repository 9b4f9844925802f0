"""Gradient norm, clipping and AdamW where a call's neighbours, its caller or
its set's shape could make it go wrong: clusters whose blocks start apart,
handles made and freed at awkward moments, the range splits of large sets.

Tolerances as derived in test_gradients.py: an L2 norm is off by 10 u of
itself, u = 2^-24, a max norm by the one product with the pre-scale."""

import math
import os
import re

import pytest

import collective_reduction_gb300 as ar
from test_gradients import U, adamw_reference, assert_close, tdt, types_of

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    return ensure_built()


def function_bodies(path):
    """{name: body} of the functions of a source file, comments taken out."""
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    out = {}
    for m in re.finditer(r"(\w+)\([^(){};]*\)(?: const)? \{\n", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        out[m.group(1)] = text[m.end():at]
    return out


# ------------------------------------------------- blocks of a cluster

def test_no_block_writes_to_another_before_it_has_started():
    """Shared memory of another block of the cluster is written only after a
    cluster barrier at which that block arrived."""
    bodies = function_bodies(os.path.join(ROOT, "collective_reduction_gb300", "csrc", "gradients.cu"))
    assert "barrier.cluster.arrive" in bodies["cluster_started"]
    users = 0
    for name, body in bodies.items():
        remote = body.find("st.shared::cluster")
        if remote >= 0:
            assert 0 <= body.find("barrier.cluster.wait") < remote, name
        if "cluster_join<" in body or "cluster_join(" in body:
            users += 1
            assert 0 <= body.find("cluster_started()") < body.find("griddep_wait()"), name
    assert users == 2  # the record's cluster and the small sets'


@gpu
@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 33, 113, 127, 128, 129, 300, 512, 513, 4000])
def test_clusters_with_blocks_that_have_nothing_to_read(n, kind):
    """Up to 128 tensors are one cluster of as many blocks as they fill; with 129
    to 512 ranges the record's cluster has seven blocks without a sum."""
    import torch
    g = torch.randn(n, generator=torch.Generator().manual_seed(n))
    views = list(torch.cat([g, g.new_zeros(3)]).cuda()[:n].split(1))
    x = g.double()
    norm = float(x.norm() if kind == "l2" else x.abs().max())
    h = ar.Grads(views, out=[torch.empty(1, device="cuda") for _ in views])
    records = torch.empty(200, 4, device="cuda")
    for k in range(0, 200, 2):
        h.norm(max_norm=0.5 * norm, kind=kind, result=records[k])
        h.clip(0.5 * norm, kind=kind, result=records[k + 1])
    got = records.cpu()
    assert bool((got == got[0]).all())
    assert_close(got[0, 0].item(), norm, 10 * U if kind == "l2" else U, "norm")
    assert_close(got[0, 1].item(), 0.5, 11 * U, "scale")
    want = g * got[0, 1]
    assert all(v.item() == w.item() for v, w in zip(h.out, want))


# ------------------------------------------------- what a call leaves behind

def test_no_load_pins_lines_in_l2():
    """Lines of a higher than usual priority outlive the call and take L2 from
    every kernel that follows."""
    bodies = function_bodies(os.path.join(ROOT, "collective_reduction_gb300", "csrc", "gradients.cu"))
    assert "createpolicy" in bodies["keep_policy"]
    assert not [name for name, body in bodies.items() if "evict_last" in body]


@gpu
def test_a_handle_that_found_no_memory_can_be_made_again():
    """The failure is reported once: with memory free again the same call works."""
    import torch
    n = 1 << 28  # a table of 32 MB
    p, g = (torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m, v = (torch.zeros(n, device="cuda") for _ in range(2))
    ar.AdamW([p[:8]], [g[:8]], [m[:8]], [v[:8]]).step(1, lr=0.0)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    filler = torch.empty(free - (20 << 20), dtype=torch.uint8, device="cuda")
    try:
        with pytest.raises(ar.ArError) as e:
            ar.AdamW([p], [g], [m], [v])
    finally:
        del filler
        torch.cuda.empty_cache()
    assert e.value.name == "AR_ERR_NOMEM"
    g.fill_(1.0)
    opt = ar.AdamW([p], [g], [m], [v])
    assert opt.info()["table_bytes"] > 20 << 20
    opt.step(1, lr=0.5)
    assert float(p.max()) == -0.5 and float(p.min()) == -0.5


@gpu
@pytest.mark.parametrize("sizes", [[0], [0] * 3000, [0] * 1000 + [1]])
def test_a_new_handle_is_complete_for_any_stream(sizes):
    """Made and used at once on a stream that waits for no other, over memory
    that held other numbers: every tensor's norm is its own."""
    import torch
    s = torch.cuda.Stream()
    x = torch.ones(1, device="cuda")
    views = [x[:n] for n in sizes]
    torch.cuda.synchronize()
    for k in range(20):
        with torch.cuda.stream(s):
            other = ar.Grads([torch.full((4096,), 7.0, device="cuda")])
            other.norm()
            other.close()  # its memory is free for the next handle
            h = ar.Grads(views)
            per = torch.full((len(sizes),), -7.0, device="cuda")
            rec = h.norm(max_norm=0.5, per_tensor=per)
        s.synchronize()
        total = float(sum(sizes))
        assert rec.tolist() == [total, 0.5 if total else 1.0, 0.0, total]
        assert per.tolist() == [float(n) for n in sizes]
        h.close()


# ------------------------------------------------- the range splits of large sets

class Large:
    """Views of guarded device buffers as test_gradients.Tensors, filled on the
    device: tensor i starts `offset` elements past a 256-byte boundary."""

    def __init__(self, sizes, types, offset=0, seed=0, sigma=1.0, square=False):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.big, self.views = [], []
        for n, t in zip(sizes, types_of(types, len(sizes))):
            big = torch.full((256 + offset + n + 256,), -7.0, dtype=tdt(t), device="cuda")
            x = torch.randn(n, generator=g, device="cuda") * sigma
            big[256 + offset:256 + offset + n] = x.square_() if square else x
            self.big.append(big)
            self.views.append(big[256 + offset:256 + offset + n])
        self.lead = 256 + offset

    def check_guards(self):
        for b, v in zip(self.big, self.views):
            assert bool((b[:self.lead] == -7.0).all()) and bool((b[self.lead + v.numel():] == -7.0).all())


# 1, 2, 4 and 8 warps to a range; several ranges to a block in place (above 120M
# float32 elements, 240M bfloat16)
LARGE = {
    "5m": [5000011, 64, 3, 100003],
    "20m": [33, 7000001, 0, 13000007],
    "130m": [130000007, 70001],
    "500m": [12289, 250000003, 251000001],
}


PAIRS = [("float32", None), ("bfloat16", None), ("mixed", None), ("float32", "float32"), ("bfloat16", "float32"),
         ("float32", "bfloat16"), ("bfloat16", "bfloat16"), ("mixed", "float32")]


@gpu
@pytest.mark.parametrize("sizes,pair,offsets",
                         [(s, p, o) for s in ("5m", "20m", "130m") for p in PAIRS
                          for o in ([(0, 0), (1, 1), (0, 1), (3, 2)] if p[1] else [(0, 0), (1, 1)])] +
                         [("500m", p, (0, 0)) for p in PAIRS[:2]])
def test_clip_of_large_sets(sizes, pair, offsets):
    import torch
    n = LARGE[sizes]
    g = Large(n, pair[0], offsets[0], seed=3)
    o = None if pair[1] is None else Large(n, pair[1], offsets[1], seed=4)
    before = [v.clone() for v in g.views]
    square = sum(float(v.double().square().sum()) for v in before)
    h = ar.Grads(g.views, out=None if o is None else o.views)
    rec = h.clip(0.25 * math.sqrt(square))
    assert_close(rec[0].item(), math.sqrt(square), 10 * U, "norm")
    assert_close(rec[1].item(), 0.25, 11 * U, "scale")
    for b, a in zip(before, (g if o is None else o).views):
        assert torch.equal(a, (b.float() * rec[1]).to(a.dtype))
    g.check_guards()
    if o is not None:
        assert all(torch.equal(a, b) for a, b in zip(g.views, before))
        o.check_guards()
    h.close()


@gpu
@pytest.mark.parametrize("offsets", [(0, 0, 0, 0, 0), (1, 1, 1, 1, 1), (0, 1, 0, 0, 0), (2, 1, 0, 3, 5)])
@pytest.mark.parametrize("kinds", [("float32", "float32", False), ("float32", "bfloat16", True),
                                   ("bfloat16", "bfloat16", False), ("mixed", "mixed", False)])
@pytest.mark.parametrize("sizes", [[1500001, 3, 5000], [5000011, 64], [20000003, 255, 0, 70001]])
def test_adamw_of_large_sets(sizes, kinds, offsets):
    import torch
    k = len(sizes)
    p = Large(sizes, kinds[0], offsets[0], seed=1, sigma=0.05)
    g = Large(sizes, kinds[1], offsets[1], seed=2, sigma=1e-2)
    m = Large(sizes, "float32", offsets[2], seed=3, sigma=3e-3)
    v = Large(sizes, "float32", offsets[3], seed=4, sigma=1e-2, square=True)
    w = Large(sizes, "bfloat16", offsets[4], seed=5) if kinds[2] else None
    before = [[a.double() for a in x.views] for x in (p, g, m, v)]
    decay = [float(1 + i % 2) for i in range(k)]
    opt = ar.AdamW(p.views, g.views, m.views, v.views, copies=w.views if w else None, decay=decay)
    record = ar.Grads(g.views).norm(max_norm=1e-2)
    opt.step(7, lr=3e-3, beta2=0.95, weight_decay=0.1, clip=record)
    for i in range(k):
        want = adamw_reference(*[b[i] for b in before], record[1].item(), 7, 3e-3, 0.9, 0.95, 1e-8, 0.1 * decay[i])
        for x, value, bound in ((p, want[0], want[3]), (m, want[1], want[4]), (v, want[2], want[5])):
            if x.views[i].dtype == torch.bfloat16:
                bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * value.abs()
            assert bool(((x.views[i].double() - value).abs() <= bound).all()), (i, sizes[i])
        if w:
            assert torch.equal(w.views[i], p.views[i].bfloat16())
        assert torch.equal(g.views[i].double(), before[1][i])
    for x in (p, g, m, v, w):
        if x:
            x.check_guards()


# ------------------------------------------------- what the binding takes

def layout_pairs():
    """Pairs of tensors whose elements lie in the same order, made in two ways."""
    import torch
    a = torch.zeros(4, 1, 3).permute(2, 1, 0)
    b = torch.zeros(4, 3).t().unsqueeze(1)
    c = torch.zeros(2, 5, 3, 1).to(memory_format=torch.channels_last)
    d = torch.zeros(2, 3, 5).permute(0, 2, 1).unsqueeze(3)
    return [(a, b), (c, d)]


@pytest.mark.parametrize("k", [0, 1])
def test_dimensions_of_size_one_do_not_tell_layouts_apart(k):
    a, b = layout_pairs()[k]
    assert a.shape == b.shape and not a.is_contiguous() and a.stride() != b.stride()
    assert ar._layout(a) == ar._layout(b) is not None


@gpu
def test_binds_equal_layouts_made_in_two_ways():
    import torch
    for a, b in layout_pairs():
        p, g, m, v = a.cuda(), b.cuda(), torch.zeros_like(a).cuda(), torch.zeros_like(b).cuda()
        g.normal_(0.0, 1.0)
        ar.AdamW([p], [g], [m], [v]).step(1, lr=0.5, beta1=0.0, beta2=0.0)
        assert torch.equal(m, g) and torch.equal(v, g * g)


# ------------------------------------------------- what autograd sees

@gpu
def test_backward_over_a_value_from_before_the_update_is_an_error():
    import torch
    w, x = torch.randn(8, 8, device="cuda", requires_grad=True), torch.randn(8, 8, device="cuda", requires_grad=True)
    low = torch.randn(8, 8, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    g, m, v = (torch.ones(8, 8, device="cuda") for _ in range(3))
    opt = ar.AdamW([w], [g], [m], [v], copies=[low])
    steps = torch.zeros(1, dtype=torch.int64, device="cuda")
    for counted in (False, True):
        saved = (x @ w).sum(), (x.bfloat16() @ low).sum()
        opt.step(steps if counted else 1, lr=0.1)
        for loss in saved:
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                loss.backward()
        (x @ w).sum().backward()  # a forward after the update is fine


@gpu
@pytest.mark.parametrize("elsewhere", [False, True])
def test_backward_over_a_gradient_from_before_the_clip_is_an_error(elsewhere):
    import torch
    g, x = torch.ones(64, device="cuda"), torch.ones(64, device="cuda", requires_grad=True)
    out = torch.ones(64, device="cuda") if elsewhere else None
    h = ar.Grads([g[:32], g[32:]], out=[out[:32], out[32:]] if elsewhere else None)
    read, written = (x * g).sum(), (x * out).sum() if elsewhere else None
    h.norm(max_norm=1.0)
    read.backward(retain_graph=True)  # a norm writes nothing
    h.clip(1.0)
    if elsewhere:
        read.backward()
        read = written
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        read.backward()


@gpu
def test_tensors_without_versions_are_taken_too():
    import torch
    with torch.inference_mode():
        p, g, m, v = (torch.zeros(8, device="cuda") for _ in range(4))
    opt = ar.AdamW([p], [g], [m], [v])
    opt.step(1, lr=0.5, weight_decay=0.5)
    ar.Grads([g]).clip(1.0)
    assert not bool(p.any())


def test_one_version_counter_is_raised_once():
    import torch
    flat, alone = torch.zeros(12), torch.zeros(3)
    owners = ar._version_owners([flat[:4], flat[4:], flat.view(3, 4), alone, alone])
    assert len(owners) == 2
    ar._version_raiser()(owners)
    assert flat._version == 1 and flat[:4]._version == 1 and alone._version == 1
    with torch.inference_mode():
        assert ar._version_owners([torch.zeros(3)]) == []


# ------------------------------------------------- freeing handles

def test_handles_wait_for_the_end_of_a_capture(monkeypatch):
    """_free against a stand-in for torch: nothing is freed while the current
    stream captures, everything with the next handle after it."""
    class Cuda:
        capturing = False

        def is_initialized(self):
            return True

        def is_current_stream_capturing(self):
            return self.capturing

    class Torch:
        cuda = Cuda()
    monkeypatch.setitem(ar.sys.modules, "torch", Torch)
    freed = []
    ar._free(freed.append, 1)
    assert freed == [1]
    Torch.cuda.capturing = True
    ar._free(freed.append, 2, keep="tensors")
    ar._free(freed.append, 3)
    ar._free()
    assert freed == [1] and [h for _, h, _ in ar._retired] == [2, 3]
    Torch.cuda.capturing = False
    ar._free()
    assert sorted(freed) == [1, 2, 3] and not ar._retired


@gpu
def test_handles_dropped_during_a_capture_do_not_end_it():
    import torch
    g = [torch.full((1000,), 2.0, device="cuda")]
    lasting, dropped = ar.Grads(g), [ar.Grads(g)]
    p, m, v = ([torch.zeros(1000, device="cuda")] for _ in range(3))
    dropped.append(ar.AdamW(p, g, m, v))
    dropped.append(ar.Plan(2, 64, "float32", "sum", "ring"))
    lasting.clip(1e9)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lasting.clip(1e9, pre_scale=0.5)
        dropped.clear()
        assert len(ar._retired) == 3
        lasting.norm()
    graph.replay()
    torch.cuda.synchronize()
    assert bool((g[0] == 1.0).all())
    ar.Grads(g).close()
    assert not ar._retired
    graph.replay()
    assert bool((g[0] == 0.5).all())


@gpu
def test_closing_twice_and_calls_after_it():
    import torch
    g = [torch.ones(8, device="cuda")]
    h = ar.Grads(g)
    h.close()
    h.close()
    with pytest.raises(ar.ArError):
        h.norm()


# ------------------------------------------------- the example in the README

def readme_alternatives():
    """The lines of README's example of a training step, once for each of its
    alternatives ("# either ...", "# or ...")."""
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read().split("After the allreduce, over lists of tensors", 1)[1].split("\n\n", 1)[1]
    lines = [x[4:] for x in re.match(r"(?:    .*\n|\n)+", text).group(0).splitlines()]
    parts = re.split(r"(?m)^# (?:either|or)\b.*$", "\n".join(x for x in lines if not x.startswith("python ")))
    return [parts[0] + p for p in parts[1:]] or parts


@gpu
def test_the_readme_example_scales_the_gradients_once():
    import torch
    assert len(readme_alternatives()) == 2
    for code in readme_alternatives():
        gen = torch.Generator(device="cuda").manual_seed(1)
        params = [torch.zeros(n, device="cuda") for n in (1000, 77)]
        for p in params:
            p.grad = torch.randn(p.shape, generator=gen, device="cuda")
        masters = [torch.randn(p.shape, generator=gen, device="cuda") for p in params]
        exp_avg = [torch.randn(p.shape, generator=gen, device="cuda") for p in params]
        exp_avg_sq = [torch.rand(p.shape, generator=gen, device="cuda") for p in params]
        before = [[x.double() for x in xs] for xs in (masters, [p.grad for p in params], exp_avg, exp_avg_sq)]
        names = {"ar": ar, "params": params, "masters": masters, "exp_avg": exp_avg, "exp_avg_sq": exp_avg_sq,
                 "bf16_weights": [p.bfloat16() for p in params], "step": 3}
        exec(code, names)
        norm = math.sqrt(sum(float(g.square().sum()) for g in before[1]))
        for i in range(2):
            want = adamw_reference(*[x[i] for x in before], 1.0 / norm, 3, 3e-4, 0.9, 0.999, 1e-8, 0.1)
            # the scale is off by 11 u, a gradient clipped in place by one more: 12 u on m (6 u by itself), 24 u on v
            # (8 u) and so 24 u on the update (16 u): within 4 times the bounds
            for got, value, bound in ((masters, want[0], want[3]), (exp_avg, want[1], want[4]),
                                      (exp_avg_sq, want[2], want[5])):
                assert bool(((got[i].double() - value).abs() <= 4 * bound).all())
