"""A sharded data-parallel training step on P virtual ranks of one GPU.

The order of FSDP / ZeRO ("All-Reduce, in depth", The APIs): every rank holds
the whole bf16 weights and its own fp32 gradient of them; the optimizer's
state -- fp32 weights and two moments -- is split over the ranks.  One step is

  1. reduce-scatter, average   rank r's gradient buffer then holds the averaged
                               gradient of the chunk that rank r owns
  2. norm                      of all owned chunks as one vector: the global
                               gradient norm, and the clip factor
  3. AdamW                     on every owned chunk, with the clip factor read
                               on the device; bf16 copies of the new weights go
                               into the owner's weight buffer
  4. all-gather                the owners' chunks to every rank

and is captured in one CUDA graph.  The model is the weights themselves: rank
r pulls them towards targets of its own, so the gradient of its loss
0.5 |w - t_r|^2 is w - t_r and the loss settles where w is the targets' mean.

With --vocab the weights are an output layer's, vocab x hidden, and every rank has
tokens of its own: their hidden states (fixed here) and next tokens, or a teacher's
top logits for them.  The gradients are then those of ar.OutputLoss, and the graph
begins with them.

    python examples/zero_step.py --ranks 8 --elements 10000019 --steps 20
    python examples/zero_step.py --ranks 4 --tokens 1000 --hidden 512 --vocab 10007 --teacher 16
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import collective_reduction_gb300 as ar  # noqa: E402


def owned(P, n):
    """[(start, stop)] of the chunk that rank r owns after the ring's
    reduce-scatter: chunk (r + 1) mod P of the ceil split of n elements."""
    size = -(-n // P)
    return [(min(n, k * size), min(n, (k + 1) * size)) for k in ((r + 1) % P for r in range(P))]


class ZeroStep:
    """P ranks' buffers and the plans and handles of one training step."""

    def __init__(self, P, n, lr=2e-2, max_norm=1.0, weight_decay=0.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.P, self.n, self.lr, self.max_norm, self.weight_decay = P, n, lr, max_norm, weight_decay
        start = 0.1 * torch.randn(n, generator=g, device="cuda")
        self.make_data(g)
        self.weights = [start.bfloat16() for _ in range(P)]
        self.grads = [torch.empty(n, device="cuda") for _ in range(P)]
        chunks = owned(P, n)
        self.master = [start[a:b].clone() for a, b in chunks]
        self.exp_avg = [torch.zeros(b - a, device="cuda") for a, b in chunks]
        self.exp_avg_sq = [torch.zeros(b - a, device="cuda") for a, b in chunks]
        grad_chunks = [x[a:b] for x, (a, b) in zip(self.grads, chunks)]
        self.scatter = ar.Plan(P, n, "float32", "avg", "ring", phase="reduce_scatter")
        self.gather = ar.Plan(P, n, "bfloat16", "sum", "ring", phase="all_gather")
        self.norm = ar.Grads(grad_chunks)
        self.adamw = ar.AdamW(self.master, grad_chunks, self.exp_avg, self.exp_avg_sq,
                              copies=[x[a:b] for x, (a, b) in zip(self.weights, chunks)])
        self.steps = torch.zeros(1, dtype=torch.int64, device="cuda")  # on the device, so that a graph counts it
        self.rate = torch.full((1,), lr, device="cuda")

    def make_data(self, g):
        self.targets = [torch.randn(self.n, generator=g, device="cuda") for _ in range(self.P)]

    def backward(self):
        """Every rank's gradient; the mean loss over ranks and elements."""
        loss = 0.0
        for w, t, g in zip(self.weights, self.targets, self.grads):
            torch.sub(w.float(), t, out=g)
            loss = loss + 0.5 * (g * g).mean()
        return loss / self.P

    def step(self):
        """Enqueue the step on the current stream; returns the norm's record."""
        self.scatter.execute(self.grads)
        record = self.norm.norm(max_norm=self.max_norm)
        self.adamw.step(self.steps, lr=self.rate, weight_decay=self.weight_decay, clip=record)
        self.gather.execute(self.weights)
        return record

    def capture(self):
        """The step as a CUDA graph: gradients in, weights out."""
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph


class OutputLayerStep(ZeroStep):
    """The step of an output layer on P ranks' tokens; `teacher`: distillation from
    so many teacher logits a token instead of cross entropy against the next one."""

    def __init__(self, P, tokens, hidden, vocab, teacher=0, **more):
        self.tokens, self.hidden, self.vocab, self.teacher = tokens, hidden, vocab, teacher
        super().__init__(P, vocab * hidden, **more)
        self.loss = ar.OutputLoss(tokens, hidden, vocab, top=teacher)
        self.records = torch.zeros(P, 4, device="cuda")  # of every rank's loss

    def make_data(self, g):
        n, v = self.tokens, self.vocab
        self.states = [torch.randn(n, self.hidden, generator=g, device="cuda").bfloat16() for _ in range(self.P)]
        self.next = [torch.randint(v, (n,), generator=g, device="cuda") for _ in range(self.P)]
        if self.teacher:
            first = torch.arange(self.teacher, device="cuda") * (v // self.teacher)
            self.ids = [(t[:, None] + first) % v for t in self.next]
            self.top = [torch.randn(n, self.teacher, generator=g, device="cuda") * 3.0 for _ in range(self.P)]

    def backward(self):
        """Every rank's gradient; the mean of the ranks' losses (on the device)."""
        for r in range(self.P):
            w, to = self.weights[r].view(self.vocab, self.hidden), self.grads[r].view(self.vocab, self.hidden)
            if self.teacher:
                self.loss.distill(self.states[r], w, self.ids[r], self.top[r], grad_weight=to, result=self.records[r])
            else:
                self.loss.cross_entropy(self.states[r], w, self.next[r], grad_weight=to, result=self.records[r])
        return self.records[:, 0].mean()

    def capture(self):
        """Losses, gradients and the step as a CUDA graph: weights in, weights out."""
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.backward()
            self.step()
        return graph


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--elements", type=int, default=10000019)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=1000, help="of a rank, with --vocab")
    ap.add_argument("--hidden", type=int, default=512, help="with --vocab")
    ap.add_argument("--vocab", type=int, default=0, help="the weights are an output layer's")
    ap.add_argument("--teacher", type=int, default=0, help="teacher logits a token, with --vocab")
    a = ap.parse_args()
    layer = a.vocab > 0
    z = OutputLayerStep(a.ranks, a.tokens, a.hidden, a.vocab, a.teacher) if layer else ZeroStep(a.ranks, a.elements)
    graph = z.capture()
    for i in range(a.steps):
        loss = None if layer else z.backward()
        graph.replay()
        if layer:
            loss = z.records[:, 0].mean()
        if i % max(1, a.steps // 10) == 0 or i == a.steps - 1:
            norm, scale, nonfinite, clipped = z.norm.record.tolist()
            print(f"step {z.steps.item():4d}  loss {loss.item():.5f}  norm {norm:10.3f}  scale {scale:.3e}"
                  f"{'  clipped' if clipped else ''}{'  skipped: nonfinite' if nonfinite else ''}")
    z.scatter.check()
    z.gather.check()
    same = all(torch.equal(z.weights[0], w) for w in z.weights[1:])
    print(f"weights of all {a.ranks} ranks equal: {same}")
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        graph.replay()
    stop.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(stop) / 20 * 1e3
    print(f"one step ({'losses, gradients, ' if layer else ''}reduce-scatter, norm, AdamW, all-gather) in a CUDA graph: {us:.1f} us")


if __name__ == "__main__":
    main()
