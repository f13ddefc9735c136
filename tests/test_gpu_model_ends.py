"""The head, norm and embedding calls together, as a training step of a tied model
uses them, and under streams and graphs.

The step: out = LN(E[id] s) gamma + beta, logp from out and E, and the gradient of
sum dlogp logp with respect to E (both uses), gamma and beta, against 64-bit autograd.
Every matrix in between is rounded to bf16, half a unit 2^-8 of each element: the
embedding's rows, out, dout and d, dx, the table's gradient twice.  Rounding of
inputs moves logits by about 2^-8 of their spread (3 here, so a logp by about 0.01 and
a p by 1 %); the sums of independent parts stay below a few of these: 4 % in norm."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


class Step:
    """The buffers of one step over `n` tokens, and its calls."""

    def __init__(self, zs, n, vocab, width, seed, dtype=BF16):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        new = lambda *s, kind=torch.float32: torch.empty(*s, dtype=kind, device="cuda")
        self.zs, self.n = zs, n
        self.table = (torch.randn(vocab, width, generator=g, device="cuda") * (3.0 / math.sqrt(width))).to(dtype)
        self.gamma = 1.0 + 0.2 * torch.randn(width, generator=g, device="cuda")
        self.beta = 0.1 * torch.randn(width, generator=g, device="cuda")
        self.ids, self.labels = new(n, kind=torch.int64), new(n, kind=torch.int64)
        self.dlogp = new(n)
        self.refill(g)
        self.x, self.y, self.dy, self.dx = (new(n, width, kind=dtype) for _ in range(4))
        self.stats, self.saved, self.logp = new(n, 2), new(n, 2), new(n)
        self.dtable = new(vocab, width, kind=dtype)
        self.dgamma, self.dbeta = new(width), new(width)
        self.head_work = zs.new_head_work(n, width, vocab)
        self.norm_work, self.embed_work = zs.new_layer_norm_work(n, width), zs.new_embed_work(n, width)
        self.ctrl = zs.new_ctrl()
        zs.zero_ctrl_init(self.ctrl, 64.0)
        self.scale = 2.0

    def refill(self, g):
        vocab = self.table.shape[0]
        self.ids.copy_(torch.randint(0, vocab, (self.n,), generator=g, device="cuda"))
        self.labels.copy_(torch.randint(0, vocab, (self.n,), generator=g, device="cuda"))
        self.labels[::5] = -100
        self.dlogp.copy_(-(torch.rand(self.n, generator=g, device="cuda") + 0.5) / self.n)

    def run(self):
        zs = self.zs
        zs.zero_embed_async(self.table, self.ids, self.x, scale=self.scale)
        zs.zero_layer_norm_async(self.x, self.gamma, self.beta, self.y, saved=self.stats)
        zs.zero_head_logp_async(self.y, self.table, self.labels, self.logp, self.head_work, saved=self.saved)
        zs.zero_head_logp_grad_async(self.y, self.table, self.labels, self.saved, self.dlogp, self.dy, self.dtable,
                                     self.head_work, ctrl_dev=self.ctrl)
        zs.zero_layer_norm_grad_async(self.dy, self.x, self.gamma, self.stats, self.dx, self.dgamma, self.dbeta, self.norm_work)
        zs.zero_embed_grad_async(self.ids, self.dx, self.dtable, self.embed_work, scale=self.scale, accumulate=True)

    def outputs(self):
        return [t.clone() for t in (self.logp, self.saved, self.dy, self.dx, self.dtable, self.dgamma, self.dbeta)]


@pytest.mark.parametrize("n,vocab,width", [(1, 300, 64), (500, 2000, 256), (1500, 5003, 768)])
def test_tied_step_against_autograd(zs, cuda_device, n, vocab, width):
    s = Step(zs, n, vocab, width, n)
    if n == 1:
        s.labels[0] = 7
    s.run()
    table, gamma, beta = (t.double().requires_grad_() for t in (s.table, s.gamma, s.beta))
    out = torch.nn.functional.layer_norm(table[s.ids] * s.scale, (width,), gamma, beta, 1e-5)
    lp = torch.log_softmax(out @ table.t(), 1)
    live = s.labels >= 0
    logp = lp[torch.arange(n, device="cuda"), s.labels.clamp(min=0)]
    (torch.where(live, logp * s.dlogp.double(), 0.0).sum() * 64.0).backward()
    assert ((s.logp.double() - torch.where(live, logp, 0.0)).abs() <= 0.1).all()
    for got, want in ((s.dtable, table.grad), (s.dgamma, gamma.grad), (s.dbeta, beta.grad)):
        assert (got.double() - want).norm() <= 0.04 * want.norm()


def test_step_in_a_graph(zs, cuda_device):
    """Captured, and replayed on other inputs: the bits of the eager calls."""
    s = Step(zs, 700, 3001, 512, 5)
    g = torch.Generator(device="cuda")
    g.manual_seed(77)
    s.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.run()
    for _ in range(3):
        s.refill(g)
        s.run()
        want = s.outputs()
        for t in (s.logp, s.saved, s.dy, s.dx, s.dtable, s.dgamma, s.dbeta):
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(s.outputs(), want))


def test_steps_on_two_streams(zs, cuda_device):
    """Two steps at once, each with its own scratch: the bits of one after the other."""
    a, b = Step(zs, 900, 4000, 256, 1), Step(zs, 300, 1500, 384, 2)
    a.run()
    b.run()
    want = a.outputs() + b.outputs()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for step, stream in zip((a, b), streams):
            with torch.cuda.stream(stream):
                step.run()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.outputs() + b.outputs(), want))


def test_given_stream(zs, cuda_device):
    """A stream given by its handle, with work before it in that stream."""
    s = Step(zs, 400, 1000, 128, 9)
    zs.zero_embed_async(s.table, s.ids, s.x)
    zs.zero_layer_norm_async(s.x, s.gamma, s.beta, s.y, saved=s.stats)
    torch.cuda.synchronize()
    want = s.y.clone()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        s.x.fill_(9.0)
        s.y.fill_(9.0)
    zs.zero_embed_async(s.table, s.ids, s.x, stream=stream)
    zs.zero_layer_norm_async(s.x, s.gamma, s.beta, s.y, stream=stream)
    stream.synchronize()
    assert torch.equal(s.y, want)


def test_example(zs, cuda_device):
    """The supervised example runs every step, repeatably, and its first gradients are autograd's."""
    import finetune_step
    mean, ctrl = finetune_step.run_supervised(steps=6, vocab=2003, width=128, tokens=360)
    again, _ = finetune_step.run_supervised(steps=6, vocab=2003, width=128, tokens=360)
    assert ctrl["step"] == 6 and ctrl["skipped"] == 0 and mean.isfinite().all() and torch.equal(mean, again)
    n, width = 360, 128
    model = finetune_step.TiedModel(2003, width, n, 3)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    ids, label = (torch.randint(0, 2003, (n,), generator=g, device="cuda") for _ in range(2))
    dlogp = -torch.rand(n, generator=g, device="cuda") / n
    ctrl = zs.new_ctrl()
    zs.zero_ctrl_init(ctrl, 256.0)
    model.gradients(ids, label, dlogp, ctrl)
    table, gamma, beta = (t.double().requires_grad_() for t in (model.table, model.master["gamma"], model.master["beta"]))
    out = torch.nn.functional.layer_norm(table[ids] * model.scale, (width,), gamma, beta, 1e-5)
    lp = torch.log_softmax(out @ table.t(), 1)[torch.arange(n, device="cuda"), label]
    ((lp * dlogp.double()).sum() * 256.0).backward()
    for got, want in ((model.grad["table"], table.grad), (model.grad["gamma"], gamma.grad), (model.grad["beta"], beta.grad)):
        assert (got.double() - want).norm() <= 0.04 * want.norm()


def test_first_calls_of_a_process_in_a_graph():
    """Captured before anything has run: nothing in a call's set-up disturbs a capture."""
    import subprocess
    code = """
import sys; sys.path[:0] = ['tests', '.']
import torch
from zero_partitioned_mixed_partition_gb300 import binding as zs
from test_gpu_model_ends import Step
s = Step(zs, 300, 700, 128, 5)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    s.run()
graph.replay()
torch.cuda.synchronize()
got = s.outputs()
s.run()
assert all(torch.equal(a, b) for a, b in zip(got, s.outputs())) and s.logp.isfinite().all()
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, (r.stdout + r.stderr)[-1500:]
