"""sel_sample16 on the GPU at borders next to a float: min-p at an id's weight, and
draws at a cumulative mass."""
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


def near_borders(x, T, least, most, many):
    """(uniform, id) pairs of a row: floats between `least` and `most` off an
    id's cumulative mass relative to the whole, and the id that they draw."""
    order = np.lexsort((np.arange(x.size), -x))
    z = x[order].astype(np.longdouble)
    w = np.exp((z - z[0]) / np.longdouble(np.float32(T)))
    cum = np.cumsum(w)
    b = cum[:-1] / cum[-1]
    u = b.astype(np.float32)
    off = np.abs(b - u.astype(np.longdouble)).astype(np.float64)
    hit = (off >= least) & (off <= most) & (u < 1)
    # both ids at the border weigh far more than the distance to it
    share = (w / cum[-1]).astype(np.float64)
    hit &= (share[:-1] > 8 * most) & (share[1:] > 8 * most)
    at = np.flatnonzero(hit)[:many]
    past = u[at].astype(np.longdouble) >= b[at]
    return u[at], order[np.where(past, at + 1, at)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind,T", [("few values", 1.0), ("few values", 0.7), ("many values", 0.9)])
def test_draws_next_to_a_cumulative_mass(dtype, kind, T):
    """Rows whose borders lie 2^-39 to 2^-35 from a float. Weights are good to
    2^-44 where they count, a sum of two float pairs to 2^-46, and about 30 of
    those lie between an id's weight and its cumulative mass, a product with
    the uniform after them: at most 2^-40 in all. A product of a float pair whose
    steps were fused would be good to 2^-24 only."""
    rng = np.random.default_rng(17)
    V = 40_000 if kind == "few values" else 9_000
    rows, us, want = [], [], []
    for _ in range(24):
        x = rng.normal(0, 1.5, size=V)
        if kind == "few values":
            x = np.round(x * 3) / 3
        x = torch.from_numpy(x).to(DT[dtype])
        u, ids = near_borders(x.double().numpy(), T, 2.0 ** -39, 2.0 ** -35, 24)
        rows += [x] * len(u)
        us.append(u)
        want.append(ids)
    us, want = np.concatenate(us), np.concatenate(want)
    assert us.size > 60
    got, _ = call(torch.stack(rows).cuda(), np.full(us.size, T, np.float32), None, None, None, us)
    assert np.array_equal(got, want), (int((got != want).sum()), us.size)
