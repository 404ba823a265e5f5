"""The operators around selection in the order a decode step runs them: hidden
states through the 4-bit head, a token per row from the 16-bit logits (or an
fp32 call), the tokens' vectors from the same 4-bit matrix."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import decode as D
from sampling_row_fp32_gb300 import binding as B

pytestmark = pytest.mark.gpu

ROWS, V, H, GROUP = 7, 20_011, 512, 64


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


class Step:
    def __init__(self, seed, rows=ROWS):
        rng = np.random.default_rng(seed)
        cuda = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.rows = rows
        self.q = cuda(rng.integers(0, 256, size=(V, H // 2), dtype=np.uint8))
        self.s = cuda(rng.uniform(0.01, 0.03, size=(V, H // GROUP))).bfloat16()
        self.z = cuda(rng.integers(6, 10, size=(V, H // GROUP), dtype=np.uint8))
        self.hidden = cuda(rng.normal(0, 1, size=(rows, H))).bfloat16()
        self.T = cuda(np.where(np.arange(rows) % 3 == 0, 0.0, 0.8).astype(np.float32))
        self.k = cuda(np.arange(rows, dtype=np.int32) * 10)
        self.p = cuda(np.full(rows, 0.95, np.float32))
        self.m = cuda(np.full(rows, 0.01, np.float32))
        self.u = cuda(rng.random(rows, dtype=np.float32))
        self.logits = torch.empty(rows, V + 5, dtype=torch.bfloat16, device="cuda")[:, :V]
        self.ids = torch.empty(rows, dtype=torch.int32, device="cuda")
        self.probs = torch.empty(rows, device="cuda")
        self.next = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda")

    def run(self, stream=None):
        B.sel_head_w4(self.hidden, self.q, self.s, self.z, GROUP, self.logits, stream)
        B.sel_sample16(self.logits, self.T, self.k, self.p, self.m, self.u, self.ids, self.probs, stream)
        B.sel_embed_w4(self.ids, self.q, self.s, self.z, GROUP, 1.5, self.next, stream)

    def check(self):
        """Ids from the logits that the head wrote, vectors of those ids."""
        n = lambda t: t.double().cpu().numpy()  # noqa: E731
        want, mag = D.head_w4(n(self.hidden), self.q.cpu().numpy(), n(self.s), self.z.cpu().numpy(), GROUP)
        # the accumulation's bound of tests/test_gpu_head.py and one rounding to bf16
        acc = (GROUP + H // GROUP + 2) * 2.0 ** -23 * mag
        got = n(self.logits)
        assert (np.abs(got - want) <= acc + 2.0 ** -8 * (np.abs(want) + acc)).all()
        ids, probs = D.sample16(got, n(self.T), self.k.cpu().numpy(), n(self.p), n(self.m), n(self.u))
        assert np.array_equal(B.ids_to_numpy(self.ids), ids)
        assert (np.abs(n(self.probs) - probs) <= 2.0 ** -24 * 1.001 * probs).all()
        rows = D.embed(ids, D.dequantise(self.q.cpu().numpy(), n(self.s), self.z.cpu().numpy(), GROUP), 1.5)
        assert (np.abs(n(self.next) - rows) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(rows)).all()


def test_step():
    s = Step(1)
    s.run()
    s.check()


def test_steps_feed_each_other_in_a_captured_graph():
    """Replays: each takes the vectors of the tokens that the one before drew."""
    s = Step(2)
    s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for _ in range(4):
        s.hidden.copy_(s.next * 30)
        s.u.copy_(torch.rand(ROWS, device="cuda"))
        for t in (s.logits, s.ids, s.probs, s.next):
            t.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        s.check()


def test_two_streams_and_two_graphs_share_nothing():
    a, b = Step(3), Step(4, rows=40)
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
    for st in (a, b):
        for t in (st.logits, st.ids, st.probs, st.next):
            t.fill_(-7)
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(sa):
            graphs[0].replay()
            a.run(sa)
        with torch.cuda.stream(sb):
            b.run(sb)
            graphs[1].replay()
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_greedy_row_equals_argmax_of_the_same_logits():
    s = Step(5)
    s.T.zero_()
    s.run()
    ids = torch.empty(ROWS, dtype=torch.int32, device="cuda")
    B.sel_argmax(s.logits.float().contiguous(), ids, B.workspace(B.SEL_OP_ARGMAX, ROWS, V))
    assert torch.equal(ids, s.ids)


def test_fp32_logits_feed_the_fp32_calls():
    s = Step(6)
    logits = torch.empty(ROWS, V, device="cuda")
    B.sel_head_w4(s.hidden, s.q, s.s, s.z, GROUP, logits)
    vals = torch.empty(ROWS, 20, device="cuda")
    ids = torch.empty(ROWS, 20, dtype=torch.int32, device="cuda")
    B.sel_topk(logits, 20, vals, ids, B.workspace(B.SEL_OP_TOPK, ROWS, V, 20))
    want, order = torch.sort(logits, dim=1, descending=True, stable=True)
    assert torch.equal(vals, want[:, :20]) and torch.equal(ids.long(), order[:, :20])


def test_a_failed_row_reaches_the_next_step_as_zeros():
    s = Step(7)
    s.hidden[2, 100] = float("nan")
    s.run()
    assert int(s.ids[2]) == -1 and torch.isnan(s.probs[2]) and not s.next[2].any()
    assert (s.ids[[0, 1, 3, 4, 5, 6]] >= 0).all()


FIRST_CALL = """
import torch
from sampling_row_fp32_gb300 import binding as B
rows, V, H = ROWS, 9001, 256
q = torch.randint(0, 256, (V, H // 2), dtype=torch.uint8, device="cuda")
s = torch.full((V, H // 64), 0.01, dtype=torch.bfloat16, device="cuda")
x = torch.randn(rows, H, device="cuda").bfloat16()
logits = torch.full((rows, V), 7.0, dtype=torch.bfloat16, device="cuda")
ids = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
probs, u = torch.empty(rows, device="cuda"), torch.rand(rows, device="cuda")
out = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    B.sel_head_w4(x, q, s, None, 64, logits)
    B.sel_sample16(logits, None, None, None, None, u, ids, probs)
    B.sel_embed_w4(ids, q, s, None, 64, 1.0, out)
g.replay()
torch.cuda.synchronize()
assert ((ids >= 0) & (ids < V)).all() and (probs > 0).all()
w = (torch.stack((q & 15, q >> 4), 2).view(V, H).float() - 8) * s.float().repeat_interleave(64, 1)
assert torch.allclose(logits.float(), x.float() @ w.t(), rtol=2.0 ** -7, atol=1e-3)
assert torch.equal(out.float(), w[ids.long()].bfloat16().float())
print("captured")
"""


@pytest.mark.parametrize("rows", [3, 40])
def test_first_call_of_a_process_inside_a_capture(rows):
    """Whatever the library asks of the driver once is allowed in a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.replace("ROWS", str(rows))], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_calls_from_two_threads():
    """Two host threads, each on its own stream with its own buffers."""
    steps = [Step(8), Step(9, rows=25)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()

    def work(i):
        for _ in range(30):
            steps[i].run(streams[i])
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for s in steps:
        s.check()


def test_binding_refuses_wrong_shapes():
    s = Step(10)
    with pytest.raises(ValueError):
        B.sel_head_w4(s.hidden[:, ::2], s.q, s.s, s.z, GROUP, s.logits)
    with pytest.raises(ValueError):
        B.sel_head_w4(s.hidden, s.q, s.s[:, :-1].contiguous(), s.z, GROUP, s.logits)
    with pytest.raises(ValueError):
        B.sel_head_w4(s.hidden, s.q, s.s.half(), s.z, GROUP, s.logits)
    with pytest.raises(ValueError):
        B.sel_head_w4(s.hidden, s.q, s.s, s.z, GROUP, s.logits[:, :-1])
    with pytest.raises(B.SelError):
        B.sel_head_w4(s.hidden, s.q, torch.empty(V, H // 16, dtype=torch.bfloat16, device="cuda"), None, 16, s.logits)
    with pytest.raises(ValueError):
        B.sel_sample16(s.logits, s.T[:-1], s.k, s.p, s.m, s.u, s.ids, s.probs)
    with pytest.raises(ValueError):
        B.sel_sample16(s.logits, s.T, s.k.float(), s.p, s.m, s.u, s.ids, s.probs)
    with pytest.raises(ValueError):
        B.sel_sample16(s.logits.t(), s.T, s.k, s.p, s.m, s.u, s.ids, s.probs)
    with pytest.raises(B.SelError):  # fp32 rows are sel_sample's
        B.sel_sample16(s.logits.float().contiguous(), s.T, s.k, s.p, s.m, s.u, s.ids, s.probs)
    with pytest.raises(ValueError):
        B.sel_embed_w4(s.ids, s.q, s.s, s.z, GROUP, 1.0, s.next[:-1])
    with pytest.raises(ValueError):
        B.sel_embed(s.ids, s.s.float()[:, :4], 1.0, s.probs)
    with pytest.raises(ValueError):
        B.sel_embed(s.ids.long(), s.s, 1.0, torch.empty(ROWS, H // GROUP, dtype=torch.bfloat16, device="cuda"))
