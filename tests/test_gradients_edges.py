"""Gradient norm, clipping and AdamW where a call's neighbours, its caller or
its set's shape could make it go wrong: clusters whose blocks start apart,
handles made and freed at awkward moments, the range splits of large sets.

Tolerances as derived in test_gradients.py: an L2 norm is off by 10 u of
itself, u = 2^-24, a max norm by the one product with the pre-scale."""

import os
import re

import pytest

import collective_reduction_gb300 as ar
from test_gradients import U, assert_close

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
