"""One allocation as the workspace of several operations: initialised again between them."""
import pytest
import torch

from oracle import learning as L
from sampling_row_fp32_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_one_allocation_for_the_heads_loss_and_selection(dtype):
    rows, V, H, k = 49, 30_001, 128, 20
    g = torch.Generator(device="cuda").manual_seed(1)
    w = (torch.randn(V, H, generator=g, device="cuda") / 4).to(dtype)
    x = torch.randn(rows, H, generator=g, device="cuda").to(dtype)
    logits = torch.randn(rows, V, generator=g, device="cuda")
    t = torch.randint(0, V, (rows,), generator=g, device="cuda").int()
    grad = torch.ones(rows, device="cuda")
    n = max(B.sel_workspace_bytes(op, rows, V, a) for op, a in ((B.SEL_OP_TOPK, k), (B.SEL_OP_ARGMAX, 0),
                                                                (B.SEL_OP_HEAD_LOSS, H), (B.SEL_OP_HEAD_LOSS_GRAD, H)))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    vals, ids, best = torch.empty(rows, k, device="cuda"), torch.empty(rows, k, dtype=torch.int32, device="cuda"), t.clone()
    want, at = torch.topk(logits, k, dim=1)
    want_loss, _ = L.head_loss(x, w, t)
    for _ in range(3):
        B.sel_workspace_init(ws)
        B.sel_head_loss(x, w, t, loss, lse, ws)  # (these two share it as it is)
        B.sel_head_loss_grad(x, w, t, lse, grad, dx, dw, ws)
        B.sel_head_loss(x, w, t, loss, lse, ws)
        B.sel_workspace_init(ws)
        B.sel_topk(logits, k, vals, ids, ws)
        B.sel_workspace_init(ws)
        B.sel_argmax(logits, best, ws)
        assert torch.equal(vals, want) and torch.equal(ids.long(), at) and torch.equal(best.long(), at[:, 0])
        assert (loss.double() - want_loss).abs().max() < 1e-4
        for got, exact in zip((dx, dw), L.head_loss_grad(x, w, t, lse, grad)):
            assert (got.double() - exact).norm() < 2.0 ** -7 * exact.norm()
