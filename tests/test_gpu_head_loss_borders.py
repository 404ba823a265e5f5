"""sel_head_loss_grad where gradients of very different sizes meet and where its inputs are
not finite, against the 64-bit formulas."""
import pytest
import torch

from oracle import learning as L
from sampling_row_fp32_gb300 import binding as B
from tests.test_gpu_head_loss import DT, NAN, logit_error, make, run_grad, run_loss

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [24, 300])
@pytest.mark.parametrize("apart", [8, 18, 20, 24, 28])
def test_rows_of_small_gradients_keep_their_bits(apart, rows, dtype):
    """Two kinds of rows, with gradients 2^apart apart and hidden states in columns of their
    own: the second half of weight_grad's columns is the small ones' alone."""
    V, H = 900, 128
    x, w, t, _ = make(apart, rows, V, H, dtype, spread=0.5)
    small = torch.arange(rows, device="cuda") % 2 == 1
    x[small, :H // 2] = 0
    x[~small, H // 2:] = 0
    x[4], t[4] = NAN, -1      # (nobody's: its size does not count either)
    x[6], t[6] = 6e4, -1
    grad = torch.where(small, 2.0 ** (12 - apart), 2.0 ** 12) * (1 + torch.arange(rows, device="cuda") % 5 / 5)
    grad[::3] *= -1
    _, lse = run_loss(x, w, t)
    dx, dw = run_grad(x, w, t, lse, grad)
    clean = torch.where(t[:, None] >= 0, x, 0.0)
    want_x, want_w = L.head_loss_grad(clean, w, t, lse.nan_to_num(), grad)
    # As in test_gpu_head_loss.check_grad: P's entries are off by their logits' error, the
    # exponential's, and half a step of the type, sums by a whole fp32 step a term, results
    # by half a step. Hidden states times their gradients are exact down to 2^-28 of the
    # largest such product and off by at most 2^-39 of twice that below.
    eps = torch.finfo(x.dtype).eps / 2
    live = (t >= 0)[:, None]
    x64, w64 = clean.double(), w.double()
    p = torch.where(live, torch.exp(x64 @ w64.T - lse.nan_to_num().double()[:, None]), 0.0)
    a = p.clone()
    at = (t >= 0).nonzero()[:, 0]
    a[at, t[at].long()] -= 1
    a = a.abs()
    dp = p * (logit_error(clean, w) + 2.0 ** -18) + a * (eps + 2.0 ** -22) + 2.0 ** -38
    g = grad.double().abs()[:, None] * live
    most = (g * x64.abs()).max()
    lost = most * 2.0 ** -38 if dtype == "f16" else most * 2.0 ** -126
    tol = (dp * g).T @ x64.abs() + (a * live).sum(dim=0)[:, None] * lost + (rows + 4) * 2.0 ** -23 * ((a * g).T @ x64.abs())
    tol = tol + eps * (want_w.abs() + tol) + torch.finfo(x.dtype).smallest_normal * eps
    half = slice(H // 2, H)
    err = (dw.double() - want_w).abs()[:, half]
    assert (err <= tol[:, half]).all(), (err / tol[:, half]).max()
    # what the rows' own targets get stands far above that bound
    mine = t[small & (t >= 0)].long()
    assert (want_w[mine][:, half].norm() > 50 * tol[mine][:, half].norm()) or apart > 24
    assert not dx[~live[:, 0]].any()
    err = (dx.double() - want_x).abs()[live[:, 0]]
    bound = g * ((dp @ w64.abs()) + (V + 300) * 2.0 ** -23 * (a @ w64.abs())) + eps * want_x.abs() * (1 + 2.0 ** -9)
    bound = bound + torch.finfo(x.dtype).smallest_normal * eps
    assert (err <= bound[live[:, 0]]).all()


def test_small_hidden_states_of_f16_keep_their_bits():
    """Subnormal hidden states times large gradients: results in f16's middle range."""
    x, w, t, grad = make(5, 40, 300, 64, "f16")
    x = (x.float() * 2.0 ** -15).half()
    grad = grad * 2.0 ** 12
    _, lse = run_loss(x, w, t)
    _, dw = run_grad(x, w, t, lse, grad)
    _, want = L.head_loss_grad(x, w, t, lse, grad)
    assert (dw.double() - want).norm() <= 2.0 ** -11 * want.norm()  # (P's rounding and the result's, each 2^-12 at most in the mean square)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [4, 260])
@pytest.mark.parametrize("lse_of", [float("inf"), -float("inf"), NAN])
def test_a_nonfinite_lse_fails_its_row(lse_of, rows, dtype):
    x, w, t, grad = make(7, rows, 500, 64, dtype, ignored=0.0)
    _, lse = run_loss(x, w, t)
    grad[2] *= -1
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[1:3] = True
    lse[bad] = lse_of
    dx, dw = run_grad(x, w, t, lse, grad)
    assert not torch.isfinite(dx[bad]).any() and torch.isfinite(dx[~bad]).all() and not torch.isfinite(dw).any()
    t[1], grad[2] = -1, 0.0  # rows that do not count may have any
    dx, dw = run_grad(x, w, t, lse, grad)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all() and not dx[bad].any()


def test_a_logit_of_minus_infinity_is_a_probability_of_zero():
    x, w, t, grad = make(8, 30, 400, 64, "bf16", ignored=0.0)
    x[:, 0] = 2.0 ** 120
    w[:, 0] = 0.0
    w[9, 0] = -2.0 ** 120  # (finite operands, a product past fp32)
    t[t == 9] = 10
    _, lse = run_loss(x, w, t)
    dx, dw = run_grad(x, w, t, lse, grad)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all() and not dw[9].any()


@pytest.mark.parametrize("rows", [5, 260])
def test_one_output_alone_is_the_same_in_f16(rows):
    """weight_grad alone has the launch for its hidden rows' exponent, hidden_grad alone has not."""
    x, w, t, grad = make(6, rows, 700, 200, "f16")
    _, lse = run_loss(x, w, t)
    dx, dw = run_grad(x, w, t, lse, grad)
    ws = B.workspace(B.SEL_OP_HEAD_LOSS_GRAD, rows, 700, 200)
    a, b = torch.full_like(x, 9.0), torch.full_like(w, 9.0)
    B.sel_head_loss_grad(x, w, t, lse, grad, a, None, ws)
    B.sel_head_loss_grad(x, w, t, lse, grad, None, b, ws)
    assert torch.equal(a, dx) and torch.equal(b, dw)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** -88, 1.0, 2.0 ** 120])
def test_hidden_states_of_zeros(size, dtype):
    """Nothing to take an exponent of: weight_grad is zeros, hidden_grad the usual."""
    x, w, t, grad = make(9, 20, 300, 64, dtype)
    x.zero_()
    grad = torch.full_like(grad, size)
    _, lse = run_loss(x, w, t)
    dx, dw = run_grad(x, w, t, lse, grad)
    assert not dw.any()
    want, _ = L.head_loss_grad(x, w, t, lse, grad)
    fits = want.abs() < torch.finfo(DT[dtype]).max / 2
    # (P's entries and the results to 2^-8, over all of which the errors lie on both sides)
    assert (dx.double() - want)[fits].norm() <= 2.0 ** -8 * want[fits].norm() + torch.finfo(DT[dtype]).smallest_normal
