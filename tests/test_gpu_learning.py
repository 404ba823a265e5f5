"""The operators that a drafter learns with, in the order a training step runs them:
the target's rows give their top logits (sel_topk), the drafter's hidden states a
cross entropy against the target's greedy tokens and its gradients, the drafter's
rows a divergence from the lists and its gradient; and what the divergence says of
the drafts' acceptance (spec_diagnostics)."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from oracle import learning as L
from sampling_row_fp32_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


class Step:
    def __init__(self, seed, rows=40, V=9001, H=256, k=20, T=1.5):
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s, dtype=torch.float32: torch.full(s, -7, dtype=dtype, device="cuda")  # noqa: E731
        self.rows, self.V, self.H, self.k, self.T = rows, V, H, k, T
        self.weight = (torch.randn(V, H, generator=g, device="cuda") * 3 / H ** 0.5).bfloat16()
        self.hidden = torch.randn(rows, H, generator=g, device="cuda").bfloat16()
        self.target = 3 * torch.randn(rows, V, generator=g, device="cuda")
        self.target[1, 5] = float("nan")  # a row that failed: no list, no target
        self.vals, self.ids = new(rows, k), new(rows, k, dtype=torch.int32)
        self.ws_topk = B.workspace(B.SEL_OP_TOPK, rows, V, k)
        self.ws = B.workspace(B.SEL_OP_HEAD_LOSS, rows, V, H)
        self.ws_grad = B.workspace(B.SEL_OP_HEAD_LOSS_GRAD, rows, V, H)
        self.loss, self.lse, self.far = new(rows), new(rows), new(rows)
        self.grad = torch.full((rows,), 1 / rows, device="cuda")
        self.dx, self.dw = torch.full_like(self.hidden, -7), torch.full_like(self.weight, -7)
        self.logits = new(rows, V + 5, dtype=torch.bfloat16)[:, :V]
        self.dlogits = new(rows, V + 3, dtype=torch.bfloat16)[:, :V]

    def run(self, stream=None):
        B.sel_topk(self.target, self.k, self.vals, self.ids, self.ws_topk, stream)
        greedy = self.ids[:, 0].contiguous()
        B.sel_head_loss(self.hidden, self.weight, greedy, self.loss, self.lse, self.ws, stream)
        B.sel_head_loss_grad(self.hidden, self.weight, greedy, self.lse, self.grad, self.dx, self.dw, self.ws_grad, stream)
        self.logits.copy_(self.hidden @ self.weight.t())
        B.sel_distill_grad(self.logits, self.vals, self.ids, None, self.T, self.grad, self.far, self.dlogits, stream)

    def wipe(self):
        for t in (self.vals, self.loss, self.lse, self.far, self.dx, self.dw, self.dlogits):
            t.fill_(-7)
        self.ids.fill_(3)

    def check(self):
        want, ids = torch.topk(torch.nan_to_num(self.target, 0.0), self.k, dim=1)
        live = torch.ones(self.rows, dtype=torch.bool, device="cuda")
        live[1] = False
        assert torch.equal(self.ids[live].long(), ids[live]) and (self.ids[1] == -1).all()
        t = self.ids[:, 0]
        loss, lse = L.head_loss(self.hidden, self.weight, t)
        # (a bf16 product's sums to fp32: far below 1e-4 at these sizes; the bounds are in the operators' tests)
        assert (self.loss.double() - loss).abs().max() < 1e-4 and (self.lse.double() - lse).abs().max() < 1e-4
        assert self.loss[1] == 0 and self.far[1] == 0 and not self.dx[1].any() and not self.dlogits[1].any()
        dx, dw = L.head_loss_grad(self.hidden, self.weight, t, self.lse, self.grad)
        for got, want in ((self.dx, dx), (self.dw, dw)):  # two roundings of 2^-9 each, of entries and of terms
            assert (got.double() - want).norm() < 2.0 ** -7 * want.norm()
        far, dl = L.distill(self.logits, self.vals, self.ids, None, self.T, self.grad)
        assert (self.far.double() - far).abs().max() < 1e-4
        assert ((self.dlogits.double() - dl).abs() <= 2.0 ** -8 * dl.abs() + 1e-9).all()


def test_step():
    s = Step(1)
    s.run()
    s.check()


def test_the_divergence_bounds_the_acceptance():
    """Over a list of the whole vocabulary the divergence is the rows' own, and bounds
    what modified rejection turns down: (1 - sum min(p, q))^2 <= D / 2 (Pinsker)."""
    S, K, V = 4, 6, 1000
    g = torch.Generator(device="cuda").manual_seed(5)
    target = 2 * torch.randn(S, K + 1, V, generator=g, device="cuda")
    draft = target[:, :K] * torch.linspace(0.1, 1.0, K, device="cuda")[:, None]
    rows, n = target[:, :K].reshape(-1, V).contiguous(), S * K
    vals, ids = torch.empty(n, V, device="cuda"), torch.empty(n, V, dtype=torch.int32, device="cuda")
    B.sel_topk(rows, V, vals, ids, B.workspace(B.SEL_OP_TOPK, n, V, V))
    far, accepted, prod = torch.empty(n, device="cuda"), torch.empty(S, K, device="cuda"), torch.empty(S, K, device="cuda")
    B.sel_distill(draft.reshape(-1, V).contiguous(), vals, ids, None, 1.0, far)
    B.spec_diagnostics(target, draft.contiguous(), 1.0, accepted, prod, B.workspace(B.SEL_OP_SPEC_DIAG, S, V, K))
    # (both to about 1e-6)
    assert ((1 - accepted).square() <= far.view(S, K) / 2 + 1e-5).all()
    assert ((1 - accepted[:, :-1]).square() > 0.1 * far.view(S, K)[:, :-1]).all()  # and is no other row's


def test_steps_in_a_captured_graph():
    s = Step(2)
    s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for i in range(3):
        s.hidden.mul_(-1.25)
        s.target[:, 7] = 20.0 + i
        s.wipe()
        g.replay()
        torch.cuda.synchronize()
        s.check()


def test_two_streams_and_two_graphs():
    """Each with buffers and workspaces of its own; eager calls of one between replays of the other."""
    a, b = Step(3), Step(4, rows=300, V=2003, H=64, k=7)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = []
    for st, stream in ((a, sa), (b, sb)):
        with torch.cuda.stream(stream):
            st.run()
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            st.run()
        graphs.append(g)
    a.wipe()
    b.wipe()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(sa):
            graphs[0].replay()
            a.run(sa)
        with torch.cuda.stream(sb):
            b.run(sb)
            graphs[1].replay()
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_calls_from_two_threads():
    steps = [Step(5), Step(6, rows=130, V=4001, H=512, k=50)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(20):
                steps[i].run(streams[i])
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for s in steps:
        s.check()


FIRST_CALL = """
import torch
from sampling_row_fp32_gb300 import binding as B
rows, V, H, k = ROWS, 3001, 64, 5
w = (torch.randn(V, H, device="cuda") / 8).half()
x = torch.randn(rows, H, device="cuda").half()
t = torch.randint(0, V, (rows,), device="cuda").int()
logits = torch.randn(rows, V, device="cuda")
vals, ids = torch.topk(torch.randn(rows, V, device="cuda"), k)
ids = ids.int()
new = lambda *s: torch.full(s, -7.0, device="cuda")
loss, lse, far, grad, dl = new(rows), new(rows), new(rows), torch.ones(rows, device="cuda"), new(rows, V)
dx, dw = torch.empty_like(x), torch.empty_like(w)
ws = B.workspace(B.SEL_OP_HEAD_LOSS, rows, V, H)
wg = B.workspace(B.SEL_OP_HEAD_LOSS_GRAD, rows, V, H)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    B.sel_head_loss(x, w, t, loss, lse, ws)
    B.sel_head_loss_grad(x, w, t, lse, grad, dx, dw, wg)
    B.sel_distill_grad(logits, vals, ids, None, 1.0, grad, far, dl)
g.replay()
torch.cuda.synchronize()
z = x.float() @ w.float().t()
p = torch.softmax(z, 1)
assert torch.allclose(loss, torch.nn.functional.cross_entropy(z, t.long(), reduction="none"), atol=1e-4)
p[torch.arange(rows), t.long()] -= 1
assert (dx.float() - p @ w.float()).norm() < 0.01 * dx.float().norm()
assert (dw.float() - p.t() @ x.float()).norm() < 0.01 * dw.float().norm()
q = torch.softmax(logits, 1)
q.scatter_add_(1, ids.long(), -torch.softmax(vals, 1))
assert torch.allclose(dl, q, atol=1e-6) and (far > 0).all()
print("captured")
"""


@pytest.mark.parametrize("rows", [3, 256, 300])
def test_first_call_of_a_process_inside_a_capture(rows):
    """Whatever the library asks of the driver once is allowed in a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.replace("ROWS", str(rows))], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
