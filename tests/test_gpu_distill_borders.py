"""sel_distill and sel_distill_grad where a sum, a reference or a rounding of theirs
could leave fp32, against the 64-bit formulas."""
import ctypes
import math
import subprocess

import pytest
import torch

from oracle import learning as L
from sampling_row_fp32_gb300 import binding as B
from tests.test_gpu_distill import DT, INF, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def named_ids(ids, V):
    named = torch.zeros(len(ids), V, dtype=torch.bool, device=ids.device)
    for r in range(len(ids)):
        at = ids[r].long()
        named[r, at[(at >= 0) & (at < V)]] = True
    return named


def bounds(x, vals, ids, lse, T, grad, want, want_x):
    """What fp32 steps may be off for rows whose listed ids hold the largest logits, with
    the teacher's lse given.

    As in test_gpu_distill.tolerances: log2(e) / T rounded stretches the logits by 2^-24,
    which moves ln q by that much of a logit's distance from the mean one, which lies
    among the listed; so ln q of a listed id is off by dq with the listed logits' width.
    ln s is the distance from the largest logit to the largest unlisted one, through two
    rounded factors and two products, and the rest as before: 2^-22 of itself and dq.
    r = 1 - sum p is off by dp, which moves r (ln r - ln s) by dp (|ln r| + |ln s| + 1),
    |ln r| below 20. A share of s is the softmax of the unlisted logits alone: off by dq
    with their own width."""
    y = x.double() / T
    V = x.shape[1]
    named = named_ids(ids, V)
    lq = torch.log_softmax(y, dim=1)
    far = lq.masked_fill(named, -INF)
    ln_s = torch.logsumexp(far, dim=1)

    def spread(keep):
        n = torch.where(keep & torch.isfinite(y), y, float("nan"))
        hi = torch.nan_to_num(n, nan=-INF).max(dim=1).values
        lo = torch.nan_to_num(n, nan=INF).min(dim=1).values
        return torch.where(hi >= lo, hi - lo, 0.0), torch.where(hi >= lo, torch.maximum(hi.abs(), lo.abs()), 0.0)
    width = spread(named)[1] + 1
    own = spread(~named & (far > ln_s[:, None] - 100))[0] + 1

    def off(w):
        depth = math.log(V) + 2 * w
        return 2.0 ** -24 * (2 * w + 2 * depth + 80) + 2.0 ** -21 + 2.0 ** -22 * depth, depth
    dq, depth = off(width)
    ds, _ = off(own)
    v = vals.double().abs().nan_to_num(posinf=0.0).max(dim=1).values / T + 1
    dp = 2.0 ** -24 * (4 * v + 40) + 2.0 ** -21 + 2.0 ** -22 * (2 * v + 8) + 2.0 ** -22 * torch.maximum(v, lse.abs().double())
    at = L._in_vocabulary(ids, V)
    p = torch.where(at >= 0, torch.exp(vals.double() / T - lse.double()[:, None]), 0.0)
    r = (1 - p.sum(dim=1)).clamp(min=0)
    size = torch.where(torch.isfinite(ln_s), ln_s.abs(), 0.0)
    loss = 3 * (dp + dq) * (2 + depth + 2 * v) + 2.0 ** -20 * (want.abs() + 1)
    loss = loss + dp * (size + 21) + r * 2.0 ** -22 * size
    T_eps = torch.finfo(x.dtype).eps / 2
    q = torch.exp(lq)
    share = torch.softmax(y.masked_fill(named, -INF), dim=1).nan_to_num(nan=0.0)
    d = q * (dq + dp)[:, None] + share * (dp + r * (2 * ds + dq + 2.0 ** -21))[:, None]
    d.scatter_add_(1, at.clamp(min=0), p * (dq + dp)[:, None] * (at >= 0))
    d = d * (grad.double().abs() / T)[:, None]
    tiny = torch.finfo(x.dtype).smallest_normal * T_eps
    # (weights below 2^-126 of a class's largest are nothing)
    return loss, d + (T_eps + 2.0 ** -22) * want_x.abs() + tiny + 2.0 ** -124 * grad.double().abs()[:, None] / T


def compare(x, vals, ids, lse, T, grad):
    want, want_x = L.distill(x, vals, ids, lse, T, grad)
    tol, tol_x = bounds(x, vals, ids, lse, T, grad, want, want_x)
    for loss, out in ((run(x, vals, ids, lse, T), None), run(x, vals, ids, lse, T, grad)):
        inf = torch.isinf(want)
        assert torch.equal(loss[inf].double(), want[inf])
        err = (loss.double() - want).abs()[~inf]
        assert (err <= tol[~inf]).all(), ((err / tol[~inf]).max(), loss, want)
        if out is not None:
            err = (out.double() - want_x).abs()
            assert (err <= tol_x).all(), (err / tol_x).max()
    return loss, out


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,V,k", [(6, 300, 9), (5, 40_001, 60), (3, 300_000, 20)])
@pytest.mark.parametrize("T,gap", [(1.0, 60.0), (1.0, 80.0), (1.0, 86.0), (1.0, 88.0), (1.0, 100.0), (0.25, 26.0), (1.0, 1e4),
                                   (4.0, 3e4)])
def test_unlisted_ids_far_below_the_list(T, gap, rows, V, k, dtype):
    """The student gives the unlisted ids next to nothing, the teacher does not: the rest's
    term is r (ln r - ln s) with s far below the smallest fp32 number, and a share of
    r of the gradient still goes to each of them."""
    x, vals, ids, lse, grad = make(int(gap), rows, V, k, dtype, T, rest=True)
    named = named_ids(ids, V)
    x -= torch.where(named, 0.0, gap).to(x.dtype)
    x[0].masked_fill_(~named[0] & (torch.arange(V, device="cuda") % 3 == 0), -INF)
    x[1].masked_fill_(~named[1], -gap)
    x[2].masked_fill_(~named[2] & (torch.arange(V, device="cuda") % 50 != 7), -INF)
    compare(x, vals, ids, lse, T, grad * (1024.0 if dtype == "f32" else 1.0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 150_000])
def test_unlisted_ids_at_the_types_lowest_value(V, dtype):
    """A mask of finfo.min on every unlisted id: ln s is that value, and their shares are even."""
    x, vals, ids, lse, grad = make(3, 5, V, 8, dtype, 2.0, rest=True)
    named = named_ids(ids, V)
    x[::2] = torch.where(named, x, torch.finfo(x.dtype).min)[::2]
    x[4] = torch.where(named[4], torch.finfo(x.dtype).min, x[4])  # and on every listed one
    want, want_x = L.distill(x, vals, ids, lse, 2.0, grad)
    loss, out = run(x, vals, ids, lse, 2.0, grad)
    # (r and the p of the listed ids are off by about 1e-5, which the distance magnifies)
    assert ((loss.double() - want).abs() <= 1e-4 * want.abs() + 1e-4).all(), (loss, want)
    assert ((out.double() - want_x).abs() <= 1e-4 * grad.double()[:, None] + 2.0 ** -8 * want_x.abs()).all()


def exhausted(seed, rows, V, some, k, T, mask):
    """Rows of which `some` ids count; the others are -Inf to the teacher and `mask` to the student."""
    g = torch.Generator().manual_seed(seed)
    teacher = torch.full((rows, V), -INF)
    x = torch.full((rows, V), mask)
    for r in range(rows):
        at = torch.randperm(V, generator=g)[:some]
        teacher[r, at] = 3 * torch.randn(some, generator=g)
        x[r, at] = 0.7 * teacher[r, at] + torch.randn(some, generator=g)
    vals, ids = torch.topk(teacher, k, dim=1)
    lse = torch.logsumexp(teacher.double() / T, dim=1).float()
    grad = 0.5 + torch.rand(rows, generator=g)
    return x.cuda(), vals.cuda(), ids.int().cuda(), lse.cuda(), grad.cuda()


@pytest.mark.parametrize("mask", [-INF, torch.finfo(torch.float32).min, -1e4])
@pytest.mark.parametrize("T", [1.0, 3.0])
@pytest.mark.parametrize("rows,V,some,k", [(200, 400, 30, 30), (200, 400, 30, 50), (64, 70_000, 300, 300), (64, 70_000, 300, 310)])
def test_lists_that_leave_nothing_out(rows, V, some, k, T, mask):
    """Constrained decoding: the list names every id that can come. 1 - sum p is then the
    rounding of the lse, above 0 in half of the rows, and what is left is masked in the
    student as well: the loss is the divergence over the list, not that rounding times
    the mask."""
    x, vals, ids, lse, grad = exhausted(some + k, rows, V, some, k, T, mask)
    p = torch.softmax(vals.double() / T, dim=1)
    lq = torch.log_softmax(x.double() / T, dim=1).gather(1, ids.long())
    want = torch.where(p > 0, p * (p.log() - lq), 0.0).sum(dim=1)
    loss, out = run(x, vals, ids, lse, T, grad)
    assert torch.equal(loss, run(x, vals, ids, lse, T))
    # The lse's rounding (2^-24 of it, below 8 here) scales p; fp32 logarithms of up to 40
    # in base 2 are off by 2^-18, and the exponentials of p by 2^-21.
    assert ((loss.double() - want).abs() <= (2.0 ** -20 + 2.0 ** -17) * (1 + want)).all(), (loss, want)
    w = torch.softmax(x.double() / T, dim=1)
    w.scatter_add_(1, ids.long(), -p)
    w = w * grad.double()[:, None] / T
    assert ((out.double() - w).abs() <= 2.0 ** -17 * grad.double()[:, None] / T).all()


def test_mass_outside_the_list_that_the_student_has_masked():
    """r is no rounding here: no student's probability left for it is an infinite divergence."""
    x, vals, ids, lse, grad = exhausted(9, 20, 500, 40, 20, 1.0, -INF)
    x[::2].masked_fill_(~named_ids(ids, 500)[::2], -INF)
    loss, out = run(x, vals, ids, lse, 1.0, grad)
    want, want_x = L.distill(x, vals, ids, lse, 1.0, grad)
    assert (loss[::2] == INF).all() and torch.isfinite(loss[1::2]).all() and torch.isfinite(out).all()
    assert ((loss.double() - want).abs() <= 2.0 ** -16 * want)[1::2].all()
    assert ((out.double() - want_x).abs() <= 2.0 ** -16 * grad.double()[:, None]).all()


def test_an_entry_without_probability_leaves_real_mass_alone():
    """A list that is no top-k list: one id of probability 0, and most of the row unnamed."""
    x, vals, ids, lse, grad = make(12, 30, 4000, 7, "f32", 1.0, rest=True)
    vals[:, 3] = -INF
    compare(x, vals, ids, lse, 1.0, grad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 150_000])
@pytest.mark.parametrize("T", [0.8, 1.0, 1.5])
@pytest.mark.parametrize("high", [False, True])
def test_listed_ids_at_the_types_lowest_value(high, T, V, dtype):
    """The student masks what the teacher lists: the loss is that id's p times a distance
    that fp32 holds in nats, but not in base 2."""
    x, vals, ids, _, grad = make(4, 6, V, 8, dtype, T)
    x[:, int(ids[5, 1])] = 0.0
    if high:
        x *= 1e7  # (references that are no whole numbers)
    for r, e in ((0, 3), (1, 0), (2, 7), (4, 5)):
        x[r, int(ids[r, e])] = torch.finfo(x.dtype).min
    vals[2, 7] = vals[2].min() - 30.0 * T  # p about 1e-13
    T = torch.tensor(T).item()
    want, want_x = L.distill(x, vals, ids, None, T, grad)
    loss, out = run(x, vals, ids, None, T, grad)
    assert torch.equal(loss, run(x, vals, ids, None, T))
    ok = want < torch.finfo(torch.float32).max  # (T below 1)
    assert ok[[2, 3, 5]].all() and (loss[~ok] == INF).all()
    # p is off by 2^-20 of itself (its logarithm, of up to 80 in base 2, by 2^-18)
    assert ((loss.double() - want).abs() <= 2.0 ** -17 * want.abs() + 1e-4)[ok].all(), (loss, want)
    # (ln q by 2^-20 of the logits' distances, which e^-distance takes back, and the type's rounding)
    assert ((out.double() - want_x).abs() <= 2.0 ** -16 * grad.double()[:, None] / T + 2.0 ** -8 * want_x.abs()).all()


@pytest.mark.parametrize("T", [2.0 ** -126, 1e-20, 1e30, 3e38])
def test_temperatures_at_the_ends_of_fp32(T):
    """Next to nothing and next to infinite: one id has all the weight, or all have the same."""
    x, vals, ids, _, grad = make(6, 4, 900, 6, "f32")
    x[0] = x[0].abs() + 1
    T = torch.tensor(T).item()
    want, want_x = L.distill(x, vals, ids, None, T, grad)
    loss, out = run(x, vals, ids, None, T, grad)
    fits = want < torch.finfo(torch.float32).max
    assert ((loss.double() - want).abs() <= 2.0 ** -18 * want.abs() + 2.0 ** -20)[fits].all() and (loss[~fits] == INF).all()
    # (of a gradient of g / T (q - p) each of the two to 2^-18, past fp32's largest infinite)
    g = grad.double()[:, None] / T
    err = torch.where(want_x.abs() < 3.4e38, (out.double() - want_x).abs(), 0.0)
    assert (err <= 2.0 ** -18 * g + 2.0 ** -23 * want_x.abs() + 2.0 ** -148).all()
    assert (out.abs()[want_x.abs() > 3.41e38] == INF).all()


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("rows,V,k", [(300, 64, 64), (300, 1000, 1000), (40, 30_000, 900)])
def test_no_divergence_is_below_zero(rows, V, k, rest):
    """A student equal to its teacher: rounding puts the sum on both sides of 0."""
    x, vals, ids, lse, grad = make(rows + k, rows, V, k, "f32", 1.0, rest=rest)
    x.scatter_(1, ids.long(), vals)
    if rest:  # the unlisted ids with the mass that the teacher gives them, spread evenly
        named = named_ids(ids, V)
        left = (1 - torch.exp(vals.double() - lse.double()[:, None]).sum(dim=1)).clamp(min=1e-30)
        even = lse.double() + torch.log(left / max(1, V - k))
        x.copy_(torch.where(named, x, even[:, None].float()))
    elif k < V:
        x.masked_fill_(~named_ids(ids, V), -INF)
    loss, _ = run(x, vals, ids, lse, 1.0, grad)
    assert torch.equal(loss, run(x, vals, ids, lse, 1.0))
    # (logarithms of up to 30 in base 2, and r's of its rounding over itself)
    assert (loss >= 0).all() and (loss <= 2.0 ** -16).all(), (loss.min(), loss.max())
    x[0, 5] = float("nan")
    assert torch.isnan(run(x, vals, ids, lse, 1.0)[0])


DROPPED = 7


@pytest.fixture(scope="module", params=[0, 1])
def dropping(request, tmp_path_factory):
    """The divergence as a library whose waits give up after some 10 ms, and in which one
    CTA never learns what row 7's list comes to: (rank of the CTA, the call)."""
    from sampling_row_fp32_gb300 import build
    out = str(tmp_path_factory.mktemp("drop") / "drop.so")
    subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-DSEL_WAIT_POLLS=50", f"-DSEL_TEST_DROP_ROW={DROPPED}",
                    f"-DSEL_TEST_DROP_RANK={request.param}", "-shared", build.CSRC + "/sel_distill.cu", "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.sel_distill_grad.argtypes = B.load().sel_distill_grad.argtypes
    lib.sel_distill_grad.restype = ctypes.c_int

    def call(x, vals, ids, grad, loss, d):
        return lib.sel_distill_grad(x.data_ptr(), {v: i for i, v in enumerate(DT.values())}[x.dtype], x.shape[0], x.shape[1],
                                    x.stride(0), vals.data_ptr(), ids.data_ptr(), vals.shape[1], None, 1.0,
                                    grad.data_ptr(), loss.data_ptr(), d.data_ptr(), d.stride(0),
                                    torch.cuda.current_stream().cuda_stream)
    return request.param, call


@pytest.mark.parametrize("rows,V,dtype,apart", [(20, 150_001, "f32", True), (700, 151_936, "bf16", False)])
def test_a_wait_that_runs_out_fails_its_rows(dropping, rows, V, dtype, apart):
    """Losses and whole gradients of every row that its cluster works on, and no other's."""
    rank, call = dropping
    x, vals, ids, _, grad = make(13, rows, V, 30, dtype, pad=5)
    want, want_x = run(x, vals, ids, None, 1.0, grad)
    for n in (rows, DROPPED, rows):  # (the first seven rows alone: nothing is dropped)
        loss = torch.full((n,), -77.0, device="cuda")
        d = torch.full((n, V + 5), 44.0, dtype=x.dtype, device="cuda")
        assert call(x[:n], vals[:n], ids[:n], grad[:n], loss, d) == B.SEL_OK
        torch.cuda.synchronize()
        bad = torch.isnan(loss)
        at = bad.nonzero()[:, 0].tolist()
        if n == DROPPED or (rank == 1 and not at and not apart):  # (many rows may have one CTA each)
            assert not at
        elif apart:
            assert at == [DROPPED]
        else:  # every row of the cluster, which takes each so-manieth
            step = at[1] - at[0]
            assert DROPPED in at and at == list(range(DROPPED % step, rows, step)) and step > 1
        assert torch.isnan(d[bad, :V]).all() and (d[:, V:] == 44.0).all()
        ok = ~bad
        if n == rows:
            assert torch.equal(loss[ok], want[ok]) and torch.equal(d[ok, :V], want_x[ok])


@pytest.mark.parametrize("lse_of", [2.0 ** 40, -2.0 ** 41, 3e38])
def test_an_lse_past_its_rounding_fails_its_row(lse_of):
    x, vals, ids, lse, grad = make(16, 5, 300, 5, "f32", rest=True)
    lse[1] = lse_of
    loss, out = run(x, vals, ids, lse, 1.0, grad)
    bad = torch.arange(5, device="cuda") == 1
    assert torch.equal(torch.isnan(loss), bad) and torch.isnan(out[1]).all() and torch.isfinite(out[~bad]).all()


def test_an_id_without_probability_far_below_the_students_largest():
    """p of 0 next to a distance past fp32 is nothing."""
    x, vals, ids, _, grad = make(15, 4, 300, 5, "f32")
    x[:, int(ids[0, 0])] = 3e38
    for r in range(4):
        x[r, int(ids[r, 4])] = torch.finfo(torch.float32).min
        vals[r, 4] = vals[r].max() - 500
    want, _ = L.distill(x, vals, ids, None, 1.0, grad)
    loss, out = run(x, vals, ids, None, 1.0, grad)
    assert torch.isfinite(out).all() and ((loss.double() - want).abs() <= 2.0 ** -18 * want).all()
