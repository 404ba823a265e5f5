"""sel_sample16 on the GPU at borders next to a float: min-p at an id's weight."""
import numpy as np
import pytest
import torch

from sampling_row_fp32_gb300 import binding as B

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def call(x, T, k, p, m, u):
    rows = x.shape[0]
    ids = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    probs = torch.full((rows,), -7.0, device="cuda")
    f = [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (T, k, p, m)]
    B.sel_sample16(x, *f, torch.from_numpy(u).cuda(), ids, probs)
    return B.ids_to_numpy(ids), probs.cpu().numpy()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T", [1.0, 0.7, 0.45, 3.0])
def test_min_p_next_to_a_weight(dtype, T):
    """Two ids, the second of weight w: it survives a min-p of the float at or
    below w, and not one of the next float."""
    rng = np.random.default_rng(int(T * 100))
    gap = torch.from_numpy(rng.uniform(0.01, 13.0 * T, size=1500)).to(DT[dtype])
    d = gap.double().numpy()
    w = np.exp(-d / np.float64(np.float32(T)))
    below = w.astype(np.float32)
    below = np.where(below.astype(np.float64) > w, np.nextafter(below, np.float32(0)), below).astype(np.float32)
    above = np.nextafter(below, np.float32(1))
    # exp in 64 bits, and the kernel's weight, are good to 2^-40 of w; no border is so near
    ok = (w - below > w * 2.0 ** -40) & (above - w > w * 2.0 ** -40)
    assert ok.sum() > 1400
    gap, w, below, above = gap[torch.from_numpy(ok)], w[ok], below[ok], above[ok]
    x = torch.stack((torch.zeros_like(gap), -gap), dim=1).cuda()
    n = w.size
    u = np.full(n, 1 - 2.0 ** -24, np.float32)  # the last survivor, as w > 2^-22
    Ts = np.full(n, T, np.float32)
    for m, last in ((below, 1), (above, 0)):
        ids, probs = call(x, Ts, None, None, m, u)
        assert (ids == last).all(), (int((ids != last).sum()), n)
        want = w / (1 + w) if last else np.ones(n)
        assert (np.abs(probs - want) <= 2.0 ** -24 * 1.001 * want).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_min_p_at_weights_far_down(dtype):
    """One id above 16,384 equal ones of a weight w from 2^-33 to 2^-20 that lies
    2^-42 to 2^-38.5 of itself from a float, which is min-p. The kernel's y =
    log2 w is good to 2^-43: its second float, up to 2^-20, rounds twice, and
    1 / T is held to 2^-49 of y; everything after y adds 2^-45."""
    rng = np.random.default_rng(5)
    n, ids = 1 << 22, 16_384
    gap = torch.from_numpy(rng.uniform(6.0, 22.0, size=n)).to(DT[dtype]).double().numpy()
    T = (gap / rng.uniform(20 * np.log(2), 33 * np.log(2), size=n)).astype(np.float32)
    w = np.exp(-gap.astype(np.longdouble) / T.astype(np.longdouble))
    m = w.astype(np.float32)
    off = ((m.astype(np.longdouble) - w) / w).astype(np.float64)
    at = np.flatnonzero((np.abs(off) > 2.0 ** -42) & (np.abs(off) < 2.0 ** -38.5))[:300]
    assert at.size > 150
    x = torch.zeros(at.size, 1 + ids, dtype=DT[dtype])
    x[:, 1:] = torch.from_numpy(-gap[at])[:, None]
    u = np.full(at.size, 1 - 2.0 ** -24, np.float32)  # the last survivors, as 16,384 w > 2^-20
    got, _ = call(x.cuda(), T[at], None, None, m[at], u)
    kept = off[at] <= 0
    assert np.array_equal(got > 0, kept), (int(((got > 0) != kept).sum()), at.size)
