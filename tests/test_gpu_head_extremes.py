"""sel_head_w4 on the GPU where hidden states and scales lie at opposite ends of
their types."""
import numpy as np
import pytest
import torch

from oracle import decode as D
from sampling_row_fp32_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def bound(mag, group, H):
    """At most group + H / group + 2 roundings of a whole fp32 step lie on a term's
    way, each of a sum no larger than the terms' magnitudes; results below fp32's
    smallest normal are not counted."""
    return (group + H // group + 2) * 2.0 ** -23 * mag + 2.0 ** -126


@pytest.mark.parametrize("rows", [1, 3, 8, 20])
@pytest.mark.parametrize("big,small,scale", [(126, 96, -127), (127, 98, -126), (126, 110, -126), (110, 80, -126), (60, 31, -60),
                                             (-90, -120, 100), (-96, -126, 110), (-100, -126, 100)])
def test_small_hidden_states_beside_unweighed_large_ones(rows, big, small, scale):
    """The large ones meet weights of zero, so that the few small ones decide, and
    the scales bring their sums back into range."""
    rng = np.random.default_rng(rows)
    V, H, group = 300, 512, 64
    q = rng.integers(0, 256, size=(V, H // 2), dtype=np.uint8)
    x = rng.uniform(1, 2, size=(rows, H)) * rng.choice([-1, 1], size=(rows, H)) * 2.0 ** small
    x[rng.random((rows, H)) < 0.95] = 0
    for k in (5, 130, 311, 480):  # nibble 8: weight 0
        x[:, k] = rng.uniform(1, 1.99, size=rows) * 2.0 ** big
        q[:, k // 2] = (q[:, k // 2] & (0xF0 if k % 2 == 0 else 0x0F)) | (8 << (4 * (k % 2)))
    x = torch.from_numpy(x).bfloat16()
    s = torch.from_numpy(rng.uniform(0.5, 1.0, size=(V, H // group)) * 2.0 ** scale).bfloat16()
    logits = torch.empty(rows, V, device="cuda")
    B.sel_head_w4(x.cuda(), torch.from_numpy(q).cuda(), s.cuda(), None, group, logits)
    want, mag = D.head_w4(x.double().numpy(), q, s.double().numpy(), None, group)
    off = np.abs(logits.double().cpu().numpy() - want)
    assert (off <= bound(mag, group, H)).all(), np.max(off / bound(mag, group, H))


@pytest.mark.parametrize("rows", [1, 8])
@pytest.mark.parametrize("x_exp,scale", [(126, -20), (126, -100), (127, -126), (120, -8)])
def test_groups_of_hidden_states_near_the_largest_float(rows, x_exp, scale):
    """Up to 8 hidden rows: a group's sum may pass the largest float where its
    product with the scale does not."""
    rng = np.random.default_rng(rows)
    V, H, group = 200, 256, 128
    q = rng.integers(0, 256, size=(V, H // 2), dtype=np.uint8)
    x = torch.from_numpy(rng.uniform(-1, 1, size=(rows, H)) * 1.98 * 2.0 ** x_exp).bfloat16()
    s = torch.from_numpy(rng.uniform(0.5, 1.0, size=(V, H // group)) * 2.0 ** scale).bfloat16()
    logits = torch.empty(rows, V, device="cuda")
    B.sel_head_w4(x.cuda(), torch.from_numpy(q).cuda(), s.cuda(), None, group, logits)
    want, mag = D.head_w4(x.double().numpy(), q, s.double().numpy(), None, group)
    off = np.abs(logits.double().cpu().numpy() - want)
    assert (off <= bound(mag, group, H)).all()
