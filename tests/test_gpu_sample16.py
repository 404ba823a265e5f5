"""sel_sample16 on the GPU against sorting each row in 64 bits. Ids must be
equal: masses are kept to about 45 bits, so a draw could differ only for a uniform
within about 1e-13 of a border, and equal weights add up exactly."""
import numpy as np
import pytest
import torch

from oracle import decode as D
from sampling_row_fp32_gb300 import binding as B

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def call(x, pol, u, pad=0, off=0):
    """x: a CPU tensor of 16-bit rows. pad: elements between the rows; off:
    elements that the first row lies past a 16-byte boundary."""
    rows, V = x.shape
    flat = torch.full((off + rows * (V + pad),), float("nan"), dtype=x.dtype, device="cuda")
    view = flat[off:].view(rows, V + pad)[:, :V]
    view.copy_(x)
    ids = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    probs = torch.full((rows,), -7.0, device="cuda")
    f = [None if p is None else torch.from_numpy(np.ascontiguousarray(p)).cuda() for p in pol]
    B.sel_sample16(view, f[0], f[1], f[2], f[3], torch.from_numpy(u).cuda(), ids, probs)
    return B.ids_to_numpy(ids), probs.cpu().numpy()


def check(x, pol, u, pad=0, off=0):
    rows = x.shape[0]
    T, k, p, m = pol
    wi, wp = D.sample16(x.double().numpy(), np.ones(rows) if T is None else T, np.zeros(rows) if k is None else k,
                        np.ones(rows) if p is None else p, np.zeros(rows) if m is None else m, u)
    gi, gp = call(x, pol, u, pad, off)
    assert np.array_equal(gi, wi), np.flatnonzero(gi != wi)[:8]
    # one rounding to fp32 (2^-24), and masses to about 2^-45
    assert np.array_equal(np.isnan(gp), np.isnan(wp))
    ok = ~np.isnan(wp)
    assert (np.abs(gp[ok] - wp[ok]) <= 2.0 ** -24 * 1.001 * wp[ok] + 2.0 ** -150).all()
    return gi, gp


def policies(rng, rows, V):
    T = np.where(rng.random(rows) < 0.15, 0.0, rng.uniform(0.2, 2.0, rows)).astype(np.float32)
    k = rng.choice([0, 0, 1, 2, 20, 40, 1000, max(1, V - 1), V, V + 5, 0xFFFFFFFF], rows).astype(np.uint32).view(np.int32)
    p = np.where(rng.random(rows) < 0.3, 1.0, rng.uniform(0.01, 1.0, rows)).astype(np.float32)
    m = np.where(rng.random(rows) < 0.5, 0.0, rng.uniform(0.0, 0.5, rows)).astype(np.float32)
    return T, k.view(np.uint32), p, m


def rows_of(rng, kind, rows, V, dtype):
    x = rng.normal(0, 3, size=(rows, V))
    if kind == "equal":
        x[:] = rng.normal(0, 3, size=(rows, 1))
    elif kind == "two":
        x = np.where(rng.random((rows, V)) < 0.5, 1.5, -0.25)
    elif kind == "zeros":
        x = np.where(rng.random((rows, V)) < 0.5, 0.0, -0.0)
    elif kind == "tiny":
        x = x * 1e-7
    elif kind == "huge":
        x = x * (1e37 if dtype == "bf16" else 5e3)
    elif kind == "masked":
        x[rng.random((rows, V)) < 0.95] = -np.inf
        x[:, V // 2] = 0.5
    elif kind == "lowest":
        x[rng.random((rows, V)) < 0.9] = torch.finfo(DT[dtype]).min
    return torch.from_numpy(x).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["normal", "equal", "two", "zeros", "tiny", "huge", "masked", "lowest"])
@pytest.mark.parametrize("rows,V,pad,off", [(40, 5001, 0, 0), (9, 40_000, 8, 3)])
def test_distributions(dtype, kind, rows, V, pad, off):
    rng = np.random.default_rng(V)
    check(rows_of(rng, kind, rows, V, dtype), policies(rng, rows, V), rng.random(rows, dtype=np.float32), pad, off)


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 8191, 8192, 65_521, 65_528, 65_529, 131_057, 151_936, 262_107, 262_117])
@pytest.mark.parametrize("rows,pad,off", [(1, 0, 0), (3, 1, 5)])
def test_widths(V, rows, pad, off):
    rng = np.random.default_rng(V + rows)
    check(rows_of(rng, "normal", rows, V, "bf16"), policies(rng, rows, V), rng.random(rows, dtype=np.float32), pad, off)


@pytest.mark.parametrize("rows", [2, 18, 20, 30, 49, 76, 77, 152, 153, 200])
def test_batches(rows):
    """Batches on either side of where the number of CTAs per row changes."""
    rng = np.random.default_rng(rows)
    x = rows_of(rng, "normal", rows, 30_011, "bf16")
    check(x, policies(rng, rows, 30_011), rng.random(rows, dtype=np.float32))


@pytest.mark.parametrize("rows", [1, 60, 160])
@pytest.mark.parametrize("kind", ["equal", "half", "zeros", "spread"])
def test_values_that_fill_a_counter(rows, kind):
    """More than 65,535 ids of one value: in one CTA's share, where a batch
    gives a row few CTAs, and in the row."""
    V = 230_003
    rng = np.random.default_rng(rows)
    x = rng.normal(0, 3, size=(rows, V))
    at = rng.permutation(V)
    if kind == "equal":
        x[:] = 1.25
    elif kind == "half":
        x[:, at[:131_072]] = 2.0
        x[:, at[131_072:200_000]] = -1.5
    elif kind == "zeros":
        x[:, at[:80_000]] = 0.0
        x[:, at[80_000:160_000]] = -0.0
    else:
        x[:, at[:65_536]] = 0.5
    check(torch.from_numpy(x).to(torch.bfloat16), policies(rng, rows, V), rng.random(rows, dtype=np.float32), 3, 1)


def test_widest_rows_in_one_cta_each():
    V, rows = B.SEL_SAMPLE16_MAX_V, 130
    rng = np.random.default_rng(10)
    x = rows_of(rng, "normal", 10, V, "f16").repeat(13, 1)
    check(x, policies(rng, rows, V), rng.random(rows, dtype=np.float32))


def test_widest_row():
    V = B.SEL_SAMPLE16_MAX_V
    rng = np.random.default_rng(9)
    x = rows_of(rng, "normal", 2, V, "f16")
    check(x, policies(rng, 2, V), rng.random(2, dtype=np.float32), 0, 7)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_finite_pattern(dtype):
    """All finite bit patterns of the type, shuffled, twice over: the fullest histogram."""
    rng = np.random.default_rng(3)
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(DT[dtype])
    x = bits[torch.isfinite(bits)]
    x = torch.stack([x.repeat(2)[torch.from_numpy(rng.permutation(2 * x.numel()))] for _ in range(4)])
    T = np.array([0.0, 1.0, 3e4, 1e36 if dtype == "bf16" else 2e4], dtype=np.float32)
    k = np.array([0, 5, 0, 70_001], dtype=np.uint32)
    check(x, (T, k, None, None), np.array([0.3, 0.9, 0.7, 0.99], dtype=np.float32))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("spread", [1e-38, 1e-7, 1.0, 1e4, 3e37])
def test_temperatures_at_the_ends(dtype, spread):
    """Temperatures from the smallest float to the largest on rows of any scale."""
    if spread in (1e-38, 3e37) and dtype == "f16":
        pytest.skip("outside f16")
    rng = np.random.default_rng(8)
    T = np.array([1e-45, 1e-42, 1.2e-38, 1e-30, 1e-5, 1.0, 1e5, 1e30, 3e38, spread, spread * 0.1, spread * 3], dtype=np.float32)
    x = torch.from_numpy(rng.normal(0, spread, size=(len(T), 3000))).to(DT[dtype])
    check(x, (T, None, np.full(len(T), 0.9, np.float32), None), rng.random(len(T), dtype=np.float32))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("late", [False, True])
def test_top_k_of_long_shares(dtype, late):
    """Batches whose rows one CTA takes, top-k on: rows that rise towards their
    end, rows whose first part is masked or has few ids, zeros of both signs as
    the k-th value, NaNs past the bound."""
    rows, V = 160, 140_003
    rng = np.random.default_rng(12)
    x = rng.normal(0, 3, size=(rows, V))
    if late:
        x += np.linspace(-30, 0, V)
    x[0:20, :60_000] = -np.inf
    x[20:30, :33_000] = -np.inf
    x[20:30, 7] = 1.0
    x[30:50] = np.where(rng.random((20, V)) < 0.5, 0.0, -0.0)
    x[30:50, rng.integers(0, V, 30)] = 5.0
    x[50, V - 1] = np.inf
    x[51, V - 2] = np.nan
    x[52, V - 3] = -np.nan
    pol = list(policies(rng, rows, V))
    pol[1] = rng.choice([1, 2, 29, 40, 1000, 30_000, 32_759, 32_760, 100_000], rows).astype(np.uint32)
    check(torch.from_numpy(x).to(DT[dtype]), tuple(pol), rng.random(rows, dtype=np.float32), 1, 2)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["ties", "rising", "falling", "late ties", "zeros"])
@pytest.mark.parametrize("rows", [60, 150])
def test_draws_past_the_first_batch(dtype, kind, rows):
    """Long shares, whose top ids lie behind the batch that bounds them: few or
    many ids over the bound, one value many times."""
    V = 200_009
    rng = np.random.default_rng(rows)
    x = rng.normal(0, 2, size=V)
    if kind == "ties":
        x = np.round(x)
    elif kind in ("rising", "falling"):
        x = np.sort(x)[:: 1 if kind == "rising" else -1]
    elif kind == "late ties":
        x[rng.choice(np.arange(60_000, V), 70, replace=False)] = 9.0
    else:
        x = -np.abs(x) - 1.0
        x[rng.choice(V, 300, replace=False)] = 0.0
        x[rng.choice(V, 300, replace=False)] = -0.0
    x = torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype]).expand(rows, V)
    T = rng.uniform(0.5, 1.5, size=rows).astype(np.float32)
    T[::10] = 0.0
    k = rng.choice([1, 2, 20, 40, 84, 90, 91, 92, 93, 400, 5000], size=rows).astype(np.uint32)
    check(x, (T, k, None, None), rng.random(rows, dtype=np.float32), 5, 3)


def test_equal_weights_at_exact_borders():
    """Every weight is 1: uniforms and top-p cuts that fall on a border go by
    rational arithmetic."""
    V, n = 4096, 1024
    x = torch.full((8, V), -np.inf).to(torch.bfloat16)
    x[:, 5:5 + 4 * n:4] = 2.0
    u = np.array([0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 0.125, 0.5, 2.0 ** -10], dtype=np.float32)
    p = np.array([1, 1, 0.5, 0.25, 0.75, 2.0 ** -10, 2.0 ** -11, 1 - 2.0 ** -24], dtype=np.float32)
    k = np.array([0, 0, 0, 512, 1, 0, 0, 0], dtype=np.uint32)
    gi, gp = call(x, (None, k, p, None), u)
    for r in range(8):
        i, pr = D.sample16_row_exact(x[r].double().numpy(), int(k[r]), float(p[r]), float(u[r]))
        assert (gi[r], gp[r]) == (i, np.float32(pr)), r


def test_draws_sweep_one_row():
    """2,000 uniforms on one row."""
    rng = np.random.default_rng(4)
    x = rows_of(rng, "normal", 1, 3001, "bf16").repeat(2000, 1)
    u = np.linspace(0, 1, 2000, endpoint=False).astype(np.float32)
    pol = (np.full(2000, 0.8, np.float32), None, np.full(2000, 0.98, np.float32), None)
    gi, _ = check(x, pol, u)
    assert len(set(gi.tolist())) > 50


def test_invalid_rows_fail_closed_alone():
    rng = np.random.default_rng(5)
    rows, V = 16, 9_001
    x = rows_of(rng, "normal", rows, V, "bf16")
    T, k, p, m = np.ones(rows, np.float32), np.zeros(rows, np.uint32), np.ones(rows, np.float32), np.zeros(rows, np.float32)
    u = rng.random(rows, dtype=np.float32)
    x[1, 8_000] = np.nan
    x[2, 0] = np.inf
    x[3, :] = -np.inf
    x[4, V - 1] = -np.nan
    u[5], u[6], u[7] = 1.0, -0.5, np.nan
    T[8], T[9], T[10] = -1.0, np.inf, np.nan
    p[11], p[12] = 0.0, 1.5
    m[13], m[14] = 1.0, np.nan
    T[7] = 0.0  # greedy rows check their uniform too
    gi, gp = check(x, (T, k, p, m), u)
    assert (gi[1:15] == 0xFFFFFFFF).all() and np.isnan(gp[1:15]).all()
    assert gi[0] < V and gi[15] < V


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [12, 156])
def test_one_bad_logit_anywhere_in_a_long_row(dtype, rows):
    """Also where a row with top-k or a greedy one only counts down to a bound."""
    V = 200_009
    rng = np.random.default_rng(rows)
    x = rows_of(rng, "normal", 12, V, dtype).repeat(rows // 12, 1)
    T, k = np.ones(rows, np.float32), np.full(rows, 40, np.uint32)
    T[1::4], k[2::4] = 0.0, 0
    bad = np.zeros(rows, bool)
    for i, at in enumerate([0, 1, 4096, 40_000, 131_071, 180_002, V - 2, V - 1]):
        r = i + 2 if rows == 12 else 15 * i + i % 4
        x[r, at] = [np.nan, np.inf, -np.nan][i % 3]
        bad[r] = True
    gi, gp = check(x, (T, k, None, None), rng.random(rows, dtype=np.float32), 3, 1)
    assert np.array_equal(gi == 0xFFFFFFFF, bad) and np.array_equal(np.isnan(gp), bad)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("largest", [-0.0, 1e-40, 5.9e-8, -5.9e-8, -1e-40, -30000.0])
def test_largest_logits_of_either_sign_and_subnormal(dtype, largest):
    """The row's maximum, to which every weight is taken."""
    rng = np.random.default_rng(21)
    x = torch.from_numpy(largest - np.abs(rng.normal(0, 1, size=(6, 3001))) * max(abs(largest), 1e-3)).to(DT[dtype])
    x[:, 1000] = largest
    T = np.array([0.0, 1.0, 0.5, 1.0, 2.0, 1e-3], np.float32)
    check(x, (T, None, None, None), rng.random(6, dtype=np.float32))


def test_absent_policies_are_off():
    rng = np.random.default_rng(6)
    x = rows_of(rng, "normal", 5, 2000, "f16")
    check(x, (None, None, None, None), rng.random(5, dtype=np.float32))


def test_no_rows():
    e = torch.empty(0, device="cuda")
    B.sel_sample16(torch.empty(0, 10, dtype=torch.float16, device="cuda"), None, None, None, None, e,
                   torch.empty(0, dtype=torch.int32, device="cuda"), e)


def test_agrees_with_sel_sample():
    """One policy for all rows with top_k > 0: the same chain as sel_sample on
    the same values in fp32."""
    rng = np.random.default_rng(7)
    rows, V = 32, 50_021
    x = rows_of(rng, "normal", rows, V, "bf16").cuda()
    u = torch.from_numpy(rng.random(rows, dtype=np.float32)).cuda()
    ids, ids16 = (torch.empty(rows, dtype=torch.int32, device="cuda") for _ in range(2))
    probs, probs16 = (torch.empty(rows, device="cuda") for _ in range(2))
    B.sel_sample(x.float(), B.SampleParams(0.7, 40, 0.9, 0.05, B.SEL_ORDER_TEMP_FIRST), u, ids, probs,
                 B.workspace(B.SEL_OP_SAMPLE, rows, V, 40))
    full = lambda v: torch.full((rows,), v, device="cuda")  # noqa: E731
    B.sel_sample16(x, full(0.7), torch.full((rows,), 40, dtype=torch.int32, device="cuda"), full(0.9), full(0.05), u, ids16, probs16)
    assert torch.equal(ids, ids16)
    # sel_sample's probabilities are fp32 sums, held to 1e-5 relative
    assert torch.allclose(probs, probs16, rtol=1e-5, atol=0)
