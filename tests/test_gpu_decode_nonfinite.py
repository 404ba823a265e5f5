"""What the selection calls make of nonfinite inputs of the 4-bit head."""
import numpy as np
import pytest
import torch

from sampling_row_fp32_gb300 import binding as B

pytestmark = pytest.mark.gpu

V, H, GROUP = 1000, 256, 64


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def inputs(rows, dtype):
    rng = np.random.default_rng(rows)
    x = torch.from_numpy(rng.uniform(0.5, 1, size=(rows, H))).to(dtype).cuda()
    q = torch.from_numpy(rng.integers(0, 256, size=(V, H // 2), dtype=np.uint8)).cuda()
    s = torch.from_numpy(rng.uniform(0.01, 0.02, size=(V, H // GROUP))).to(dtype).cuda()
    return x, q, s


def head_and_sample(x, q, s):
    rows = x.shape[0]
    logits = torch.empty(rows, V, dtype=x.dtype, device="cuda")
    full = torch.empty(rows, V, device="cuda")
    ids, ids32 = (torch.full((rows,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    probs, u = torch.empty(rows, device="cuda"), torch.linspace(0, 0.99, rows, device="cuda")
    B.sel_head_w4(x, q, s, None, GROUP, logits)
    B.sel_head_w4(x, q, s, None, GROUP, full)
    B.sel_sample16(logits, None, None, None, None, u, ids, probs)
    B.sel_argmax(full, ids32, B.workspace(B.SEL_OP_ARGMAX, rows, V))
    return logits, ids.cpu(), ids32.cpu()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [4, 20])
@pytest.mark.parametrize("low", [False, True])
def test_nonfinite_hidden_states_fail_their_rows(dtype, rows, low):
    """low: the column's weights are all negative, so that +Inf gives -Inf logits only."""
    x, q, s = inputs(rows, dtype)
    if low:
        q[:, 35] &= 0xF7  # column 70 under 8
        q[:, 35] = torch.where((q[:, 35] & 15) == 8, q[:, 35] - 1, q[:, 35])
    x[1, 70], x[2, 70], x[3, 70] = float("inf"), -float("inf"), float("nan")
    logits, ids, ids32 = head_and_sample(x, q, s)
    assert not torch.isfinite(logits[1:4]).any()
    if low:
        assert (logits[1] == -float("inf")).all()
    assert (ids[1:4] == -1).all() and (ids32[1:4] == -1).all()
    rest = [r for r in range(rows) if not 1 <= r < 4]
    assert (ids[rest] >= 0).all() and (ids32[rest] >= 0).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [4, 20])
def test_a_logit_of_minus_infinity_is_a_masked_id_to_sel_sample16_only(dtype, rows):
    x, q, s = inputs(rows, dtype)
    q[77] = 0x22  # weights of -6: the matrix row's logits are -Inf
    s[77, 1] = float("inf")
    logits, ids, ids32 = head_and_sample(x, q, s)
    assert (logits[:, 77] == -float("inf")).all() and torch.isfinite(logits[:, 78:]).all()
    assert ((ids >= 0) & (ids != 77)).all()
    assert (ids32 == -1).all()
    q[77] = 0xBB  # weights of 3: +Inf
    _, ids, ids32 = head_and_sample(x, q, s)
    assert (ids == -1).all() and (ids32 == -1).all()
