"""The operators that a drafter learns with, without a GPU, at the borders of their
contracts: the 64-bit forms there, and what the library's checks let through."""
import ctypes
import math

import torch

from oracle import learning as L
from sampling_row_fp32_gb300 import binding as B
from tests.test_learning_host import lib, needs_nvcc  # noqa: F401

INF = float("inf")


def test_distill_of_unlisted_ids_far_below_the_list():
    """One id listed with p = 1/4, three others that lie 10^4 below it: s = 3 e^-10000, and
    each of them gets a third of -r."""
    x = torch.tensor([[0.0, -1e4, -1e4, -1e4]], dtype=torch.float64)
    lse = torch.tensor([math.log(4.0)], dtype=torch.float64)
    one = torch.ones(1, dtype=torch.float64)
    loss, d = L.distill(x, torch.zeros(1, 1), torch.tensor([[0]]), lse, 1.0, one)
    want = 0.25 * math.log(0.25) + 0.75 * (math.log(0.75) - (math.log(3.0) - 1e4))
    assert abs(loss.item() / want - 1) < 1e-12
    assert torch.allclose(d, torch.tensor([[0.75, -0.25, -0.25, -0.25]], dtype=torch.float64), rtol=1e-12)
    x[0, 2:] = -INF
    _, d = L.distill(x, torch.zeros(1, 1), torch.tensor([[0]]), lse, 1.0, one)
    assert torch.allclose(d, torch.tensor([[0.75, -0.75, 0, 0]], dtype=torch.float64), rtol=1e-12)


def test_distill_of_lists_that_leave_nothing_out():
    """The rounding of a 32-bit lse is no probability, where nothing is left for it."""
    v = torch.tensor([[1.0, 0.5, -INF]])
    exact = torch.logsumexp(v.double(), 1)
    x = torch.tensor([[0.3, 0.1, -INF, -INF, -INF]], dtype=torch.float64)
    want = L.distill(x[:, :3], v, torch.tensor([[0, 1, 2]]), None, 1.0)
    for lse in (exact + 3e-7, exact - 3e-7):
        for k in (2, 3):
            assert abs((L.distill(x, v[:, :k], torch.tensor([[0, 1, 2]])[:, :k], lse, 1.0) - want).item()) < 1e-6
    assert L.distill(x, v[:, :2], torch.tensor([[0, 1]]), exact + 0.1, 1.0).item() == INF
    x[0, 3] = 0.0  # (and where something is, it counts)
    _, d = L.distill(x, v[:, :2], torch.tensor([[0, 1]]), exact + 3e-7, 1.0, torch.ones(1))
    assert abs(d.sum().item()) < 1e-12


@needs_nvcc
def test_temperatures_that_are_no_normal_numbers_are_refused(lib):
    F, vp = 0x10000, ctypes.c_void_p
    for T in (1e-45, 2e-39, 1.1754942e-38):
        assert lib.sel_distill(vp(F), B.SEL_F32, 3, 10, 10, vp(F), vp(F), 4, None, T, vp(F), None) == B.SEL_EINVAL
        assert lib.sel_distill_grad(vp(F), B.SEL_F32, 3, 10, 10, vp(F), vp(F), 4, None, T, vp(F), vp(F), vp(2 * F), 10,
                                    None) == B.SEL_EINVAL
    # (the smallest that is: no rows, so that nothing is launched)
    assert lib.sel_distill(vp(F), B.SEL_F32, 0, 10, 10, vp(F), vp(F), 4, None, 2.0 ** -126, vp(F), None) == B.SEL_OK


@needs_nvcc
def test_hidden_grad_alone_of_no_rows(lib):
    """An empty tensor has no address, so the call gets NULL for both gradients."""
    F, vp = 0x10000, ctypes.c_void_p
    assert lib.sel_head_loss_grad(None, 0, vp(F), B.SEL_BF16, 10, 16, None, None, None, None, None, None, 0, None) == B.SEL_OK
    assert lib.sel_head_loss_grad(vp(F), 1, vp(F), B.SEL_BF16, 10, 16, vp(F), vp(F), vp(F), None, None, vp(F), 1 << 40,
                                  None) == B.SEL_EINVAL
