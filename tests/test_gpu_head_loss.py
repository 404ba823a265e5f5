"""sel_head_loss and sel_head_loss_grad on the GPU against the 64-bit formulas."""
import numpy as np
import pytest
import torch

from oracle import learning as L
from sampling_row_fp32_gb300 import binding as B

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def make(seed, rows, V, H, dtype, spread=2.0, ignored=0.2):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(V, H, generator=g) * spread / H ** 0.5).to(DT[dtype])
    t = torch.randint(0, V, (rows,), generator=g)
    x = torch.randn(rows, H, generator=g)
    x[::2] += 4.0 * torch.rand((rows + 1) // 2, 1, generator=g) * w[t[::2]].float()  # rows that know their token
    t = torch.where(torch.rand(rows, generator=g) < ignored, -1, t)
    grad = (0.5 + torch.rand(rows, generator=g)) * (256.0 if dtype == "f16" else 1.0)
    return x.to(DT[dtype]).cuda(), w.cuda(), t.to(torch.int32).cuda(), grad.cuda()


def run_loss(x, w, t, stream=None, ws=None):
    rows, V, H = x.shape[0], w.shape[0], x.shape[1]
    ws = B.workspace(B.SEL_OP_HEAD_LOSS, rows, V, H) if ws is None else ws
    loss, lse = (torch.full((rows,), -77.0, device="cuda") for _ in range(2))
    B.sel_head_loss(x, w, t, loss, lse, ws, stream)
    return loss, lse


def run_grad(x, w, t, lse, grad, ws=None):
    rows, V, H = x.shape[0], w.shape[0], x.shape[1]
    ws = B.workspace(B.SEL_OP_HEAD_LOSS_GRAD, rows, V, H) if ws is None else ws
    dx, dw = torch.full_like(x, -77.0), torch.full_like(w, -77.0)
    B.sel_head_loss_grad(x, w, t, lse, grad, dx, dw, ws)
    assert int(ws[:4].view(torch.int32).item()) == 0
    return dx, dw


def logit_error(x, w):
    """Of each row, the most a logit may be off: products are exact in fp32, and at
    most H + 2 roundings lie on a term's way, each a whole fp32 step (2^-23, as a
    truncating accumulator gives) of a sum no larger than the terms' magnitudes."""
    mag = x.double().abs() @ w.double().abs().T
    return (x.shape[1] + 2) * 2.0 ** -23 * mag


def check_loss(x, w, t):
    loss, lse = run_loss(x, w, t)
    want, want_lse = L.head_loss(x, w, t)
    dz = logit_error(x, w).max(dim=1).values
    # The statistics: each weight has an exponent rounded to 2^-24 of itself (which
    # counts as it shrinks, at most 2^-23) and 2^-22 of the exponential; a sum of 32 in
    # four runs, over four chunks, adds 15 roundings, the joins are finer: below 2^-19.
    # A loss moves by 1 - exp(-loss) times what the difference of its logits does.
    d = 2 * dz + 2.0 ** -19
    tol = (1 - torch.exp(-want)) * d * (1 + d) + 2.0 ** -23 * want + 2.0 ** -126
    err = (loss.double() - want).abs()
    assert (err <= tol).all(), (err / tol).max()
    err = (lse.double() - want_lse).abs()
    tol = dz + 2.0 ** -19 + 2.0 ** -23 * want_lse.abs()
    assert (err <= tol).all(), (err / tol).max()
    return loss, lse


def check_grad(x, w, t, lse, grad):
    dx, dw = run_grad(x, w, t, lse, grad)
    want_x, want_w = L.head_loss_grad(x, w, t, lse, grad)
    T = x.dtype
    eps = torch.finfo(T).eps / 2
    V, rows = w.shape[0], x.shape[0]
    x64, w64, l64 = x.double(), w.double(), lse.double()
    tl = t.long()
    live = (tl >= 0) & (tl < V) & (grad != 0)
    p = torch.exp(x64 @ w64.T - l64[:, None])
    p[~live] = 0
    # An entry of P: its logit's error and that of the exponential (its exponent, z -
    # lse rounded, moves it by 2^-23 |z - lse|, and |d| e^d <= 1 below), the same on
    # the target's e^d - 1, whose own rounding and that to T come on top; f16 holds it
    # 2^14 up, where 2^-25 is half its smallest step.
    dz = logit_error(x, w) + 2.0 ** -20
    depth = 1 + (x64 @ w64.T - l64[:, None]).abs()
    dp = p * (dz + 2.0 ** -23 * depth) * (1 + 2.0 ** -8)
    hot = torch.zeros_like(p)
    hot[live, tl[live]] = 1.0
    a = (p - hot).abs()
    dp = dp + a * (eps + 2.0 ** -22) + (2.0 ** -39 if T == torch.float16 else 2.0 ** -134) * live[:, None]
    g = grad.double().abs() * live
    # sums: a rounding of a whole fp32 step for each term, as above
    mag = (a + dp) @ w64.abs()
    tol = g[:, None] * (dp @ w64.abs() + (V + 300) * 2.0 ** -23 * mag)
    tiny = torch.finfo(T).smallest_normal * eps
    tol = tol + eps * (want_x.abs() + tol) + tiny
    err = (dx.double() - want_x).abs()
    assert (err <= tol).all(), (err / tol).max()
    assert not dx[~live].any()
    # hidden rows times grad / max grad, rounded to T once more, unless the ratio is 1
    top = g.max()
    ratio = torch.where(g == top, 0.0, eps + 2.0 ** -23)
    u = x64.abs() * (1 + ratio[:, None])
    du = x64.abs() * ratio[:, None] + torch.where(g == top, 0.0, tiny * (1 + top / g.clamp(min=1e-300)))[:, None] * live[:, None]
    ga, gd = a * g[:, None], dp * g[:, None]
    tol = gd.T @ u + ga.T @ du + gd.T @ du
    tol = tol + (rows + 4) * 2.0 ** -23 * ((ga + gd).T @ u)
    tol = tol + eps * (want_w.abs() + tol) + tiny
    err = (dw.double() - want_w).abs()
    assert (err <= tol).all(), (err / tol).max()
    return dx, dw


SHAPES = [(1, 1, 8), (1, 300, 64), (2, 129, 72), (31, 256, 128), (49, 1000, 264), (127, 257, 520), (128, 512, 64),
          (129, 513, 64), (200, 127, 136), (256, 1031, 512), (257, 2, 40), (300, 3001, 1000), (600, 700, 2880)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,V,H", SHAPES)
def test_loss(rows, V, H, dtype):
    x, w, t, _ = make(rows + V, rows, V, H, dtype)
    check_loss(x, w, t)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,V,H", SHAPES)
def test_grad(rows, V, H, dtype):
    x, w, t, grad = make(rows + V, rows, V, H, dtype)
    _, lse = run_loss(x, w, t)
    check_grad(x, w, t, lse, grad)
