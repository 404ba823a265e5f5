"""sel_distill and sel_distill_grad on the GPU against the 64-bit formulas."""
import pytest
import torch

from oracle import learning as L
from sampling_row_fp32_gb300 import binding as B

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def make(seed, rows, V, k, dtype, T=1.0, pad=0, rest=False, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    teacher = torch.randn(rows, V, generator=g) * spread
    teacher[::2, V // 3] += 6.0  # every other row peaked
    x = (0.7 * teacher + torch.randn(rows, V, generator=g)).to(DT[dtype])
    vals, ids = torch.topk(teacher, k, dim=1)
    order = torch.argsort(torch.rand(rows, k, generator=g), dim=1)  # lists come in any order
    vals, ids = vals.gather(1, order), ids.gather(1, order).to(torch.int32)
    lse = torch.logsumexp(teacher.double() / T, dim=1).float() if rest else None
    buf = torch.full((rows, V + pad), NAN, dtype=DT[dtype], device="cuda")
    buf[:, :V] = x.cuda()
    grad = 0.5 + torch.rand(rows, generator=g)
    return buf[:, :V], vals.cuda(), ids.cuda(), None if lse is None else lse.cuda(), grad.cuda()


def run(x, vals, ids, lse, T, grad=None, out=None, loss=True, stream=None):
    rows = x.shape[0]
    got = torch.full((rows,), -77.0, device="cuda") if loss else None
    if grad is None:
        B.sel_distill(x, vals, ids, lse, T, got, stream)
        return got
    if out is None:
        out = torch.full((rows, x.shape[1]), -77.0, dtype=x.dtype, device="cuda")
    B.sel_distill_grad(x, vals, ids, lse, T, grad, got, out, stream)
    return got, out


def tolerances(x, vals, ids, lse, T, grad, want, want_x):
    """Bounds of what the fp32 steps may be off (a unit of 2^-24 is half a step).

    A weight 2^(x kf - m): kf = log2(e) / T rounded stretches the row's logits by
    2^-24, which moves ln q_j by 2^-24 of its distance from the mean logit; the
    exponent's own rounding by 2^-24 of its size; the exponential by 2^-22. The
    sums of 2^-24 a term of a thread's run (up to 64 here) and of a vector's eight:
    together ln q and ln p are off by at most dq, dp below; every logarithm that
    comes on top is rounded to 2^-23 of itself."""
    y = x.double() / T
    finite = torch.isfinite(y)
    width = torch.where(finite, y, 0.0).abs().max(dim=1).values + 1
    depth = torch.log(torch.tensor(float(x.shape[1]))) + 2 * width
    dq = 2.0 ** -24 * (2 * width + 2 * depth + 80) + 2.0 ** -21 + 2.0 ** -22 * depth
    v = torch.where(torch.isfinite(vals), vals.double(), 0.0).abs().max(dim=1).values / T + 1
    big = v if lse is None else torch.maximum(v, lse.abs().double())
    dp = 2.0 ** -24 * (4 * v + 40) + 2.0 ** -21 + 2.0 ** -22 * (2 * v + 8) + (0 if lse is None else 2.0 ** -24 * 4 * big)
    # each term p (ln p - ln q) by dp of p, and its difference by dp + dq; p sums to at
    # most about 1, and |ln p - ln q| to at most depth + 2 v; the class of the rest
    # likewise, its r = 1 - sum p by dp: ln r - ln s moves by dp / r, times r
    one = (dp + dq) * (2 + depth + 2 * v) + 2.0 ** -21 * (want.abs() + 1)
    loss = one if lse is None else 3 * one
    T_eps = torch.finfo(x.dtype).eps / 2
    tol = None
    if want_x is not None:
        g = grad.double().abs() / T
        q = torch.softmax(y, dim=1)
        at = L._in_vocabulary(ids, x.shape[1])
        p = torch.zeros_like(q)
        L_ = torch.logsumexp(torch.where(at >= 0, vals.double() / T, -INF), dim=1) if lse is None else lse.double()
        pv = torch.where(at >= 0, torch.exp(vals.double() / T - L_[:, None]), 0.0)
        p.scatter_add_(1, at.clamp(min=0), pv)
        d = (q + p) * (dq + dp)[:, None]
        if lse is not None:  # r / s times q: r by dp, s relatively by dq
            named = torch.zeros_like(q, dtype=torch.bool)
            for r in range(len(at)):
                named[r, at[r][at[r] >= 0]] = True
            s = q.masked_fill(named, 0.0).sum(dim=1)
            r = (1 - pv.sum(dim=1)).clamp(min=0)
            d = d + q.masked_fill(named, 0.0) * ((dp + r * dq * 2 + r * 2.0 ** -22) / s.clamp(min=1e-300))[:, None]
        d = d * g[:, None]
        tiny = torch.finfo(x.dtype).smallest_normal * T_eps
        tol = d + (T_eps + 2.0 ** -22) * want_x.abs() + tiny + 2.0 ** -126
    return loss, tol


def check(x, vals, ids, lse, T, grad):
    want, want_x = L.distill(x, vals, ids, lse, T, grad)
    tol, tol_x = tolerances(x, vals, ids, lse, T, grad, want, want_x)
    nan = torch.isnan(want)
    for got in (run(x, vals, ids, lse, T), None):
        if got is None:
            got, out = run(x, vals, ids, lse, T, grad)
        assert torch.equal(torch.isnan(got), nan)
        inf = torch.isinf(want)
        assert torch.equal(got[inf].double(), want[inf])
        err = (got.double() - want).abs()
        ok = ~nan & ~inf
        assert (err <= tol)[ok].all(), (err / tol)[ok].max()
    nan = torch.isnan(want_x)
    assert torch.equal(torch.isnan(out), nan)
    err = (out.double() - want_x).abs()
    assert (err <= tol_x)[~nan].all(), (err / tol_x)[~nan].max()
    return got, out


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("rows,V,k,pad", [
    (1, 1, 1, 0), (1, 2, 1, 0), (3, 7, 7, 0), (2, 100, 5, 3), (5, 1000, 64, 0), (7, 4097, 20, 1), (4, 9001, 1024, 0),
    (40, 5003, 513, 5), (3, 33_001, 100, 8), (9, 65_536, 200, 0), (2, 151_936, 20, 0), (3, 248_320, 1000, 0)])
def test_shapes(rows, V, k, pad, rest, dtype):
    x, vals, ids, lse, grad = make(rows + V, rows, V, k, dtype, 1.0, pad, rest)
    check(x, vals, ids, lse, 1.0, grad)


@pytest.mark.parametrize("T", [0.3, 0.7, 1.5, 4.0, 1000.0])
@pytest.mark.parametrize("rest", [False, True])
def test_temperatures(T, rest):
    T = torch.tensor(T).item()
    x, vals, ids, lse, grad = make(5, 6, 3001, 50, "f32", T, 0, rest)
    check(x, vals, ids, lse, T, grad)


def test_many_rows_of_one_cta():
    x, vals, ids, lse, grad = make(8, 2000, 3001, 10, "bf16")
    check(x, vals, ids, lse, 1.0, grad)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,V,k", [(3, 400_001, 20), (2, 1 << 20, 1000), (600, 40_001, 7), (9, 130_000, 3)])
def test_shares_longer_than_the_ring_and_many_rounds(rows, V, k, dtype):
    x, vals, ids, lse, grad = make(rows, rows, V, k, dtype, rest=True)
    check(x, vals, ids, lse, 1.0, grad)


def test_ignored_rows_first_last_and_between():
    """More rows than run at a time, most of them without a list."""
    rows, V = 700, 20_003
    x, vals, ids, _, grad = make(1, rows, V, 12, "f16")
    ids[torch.rand(rows, device="cuda") < 0.6] = -1
    ids[:5] = -1
    ids[-3:] = -1
    vals[ids < 0] = NAN  # as sel_topk leaves a failed row
    x[2], x[-1] = NAN, INF
    check_ignored(x, vals, ids, grad)


def check_ignored(x, vals, ids, grad):
    gone = (ids < 0).all(dim=1)
    loss, out = run(x, vals, ids, None, 1.0, grad)
    assert not loss[gone].any() and not out[gone].any()
    keep = ~gone
    x, vals, ids, grad = x[keep], vals[keep], ids[keep], grad[keep]
    check(x, vals, ids, None, 1.0, grad)
    # in the whole batch a row may be split otherwise, so that its sums meet in another order
    want, want_x = L.distill(x, vals, ids, None, 1.0, grad)
    tol, tol_x = tolerances(x, vals, ids, None, 1.0, grad, want, want_x)
    assert ((loss[keep].double() - want).abs() <= tol).all() and ((out[keep].double() - want_x).abs() <= tol_x).all()


@pytest.mark.parametrize("rest", [False, True])
def test_short_lists(rest):
    """Entries without an id, anywhere in a list, whatever their values."""
    x, vals, ids, lse, grad = make(2, 50, 2000, 40, "bf16", rest=rest)
    drop = torch.rand(50, 40, device="cuda") < 0.3
    drop[:, 0] = False
    ids[drop] = 2000 + torch.randint(0, 1000, (int(drop.sum()),), device="cuda", dtype=torch.int32)
    vals[drop] = torch.where(torch.rand(int(drop.sum()), device="cuda") < 0.5, NAN, 1e30)
    ids[3, 1] = -1
    clean = torch.where(ids.long().cpu() < 2000, vals.cpu(), 0.0).cuda()
    want, want_x = L.distill(x, clean, ids, lse, 1.0, grad)
    tol, tol_x = tolerances(x, clean, ids, lse, 1.0, grad, want, want_x)
    loss, out = run(x, vals, ids, lse, 1.0, grad)
    assert ((loss.double() - want).abs() <= tol).all() and ((out.double() - want_x).abs() <= tol_x).all()


def test_rows_that_leave_nothing_or_fail():
    rows, V, k = 16, 5000, 6
    for dtype in ("f32", "f16", "bf16"):
        x, vals, ids, lse, grad = make(3, rows, V, k, dtype, rest=True)
        ids[0] = -1                  # no list
        vals[1] = -INF               # a list of nothing
        ids[2, 3] = ids[2, 5]        # an id twice
        x[3, 17] = NAN
        x[4, int(ids[4, 0])] = NAN
        x[5, 4999] = INF
        x[6] = -INF                  # every id masked
        vals[7, 2] = NAN
        vals[8, 2] = INF
        lse[9] = NAN
        lse[10] = INF
        grad[11] = 0.0
        vals[12, 1:] = -INF          # one entry counts
        x[13, :4000] = -INF          # masked ids, some of them listed
        grad[3] = 0.0
        for given in (None, lse):
            loss, out = run(x, vals, ids, given, 1.0, grad)
            bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
            bad[2:9] = True
            if given is not None:
                bad[9:11] = True
            assert torch.equal(torch.isnan(loss), bad), (dtype, loss)
            assert torch.equal(loss, run(x, vals, ids, given, 1.0)) or torch.equal(torch.nan_to_num(loss, 5.0), torch.nan_to_num(run(x, vals, ids, given, 1.0), 5.0))
            assert not loss[:2].any() and not out[:2].any() and not out[11].any() and not out[3].any()
            nan = torch.isnan(out).all(dim=1)
            bad[3] = False  # (its grad is 0)
            assert torch.equal(nan, bad), dtype
            assert torch.isfinite(out[[0, 1, 3, 11, 12, 14, 15]]).all()
            masked = (x[13] == -INF).nonzero()[:, 0]
            listed = torch.isin(masked, ids[13].long())
            assert not out[13, masked[~listed]].any()
            assert loss[13] == INF if listed.any() else torch.isfinite(loss[13])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("C", [300, 60_000])
def test_masks_of_the_types_lowest_value(dtype, C):
    """finfo.min for a mask: no weight, next to any other id; a row of nothing else is even."""
    low = torch.finfo(DT[dtype]).min
    x, vals, ids, lse, grad = make(4, 6, C, 5, dtype, 0.75, rest=True)
    named = torch.zeros(6, C, dtype=torch.bool, device="cuda")
    named.scatter_(1, ids.long(), True)
    mask = (torch.rand(6, C, device="cuda") < 0.9) & ~named
    x[mask] = low
    check(x, vals, ids, lse, 0.75, grad)
    x[2] = low
    loss, out = run(x, vals, ids, None, 0.75, grad)
    want, want_x = L.distill(x, vals, ids, None, 0.75, grad)
    assert abs(loss[2].item() - want[2].item()) <= 1e-5 * want[2].item()
    assert torch.allclose(out[2].double(), want_x[2], rtol=2.0 ** -7, atol=1e-9)


@pytest.mark.parametrize("scale", [1e3, 1e6, 1e9, 1e30])
def test_logits_of_any_size(scale):
    """Rows whose largest logit takes all: the loss is the distance to it."""
    x, vals, ids, _, grad = make(5, 5, 3000, 8, "f32")
    x = x * scale
    x[4] = -x[4].abs()
    loss, out = run(x, vals, ids, None, 1.0, grad)
    want, want_x = L.distill(x, vals, ids, None, 1.0, grad)
    # ln q is a difference of logits, times log2(e) rounded and back
    assert ((loss.double() - want).abs() <= 2.0 ** -20 * want.abs() + 1e-5).all()
    # (a weight's exponent is off by 2^-24 of itself, and |d| e^-d is below 1)
    assert ((out.double() - want_x).abs() <= 2.0 ** -20 * want_x.abs() + 2.0 ** -20 * grad.double()[:, None]).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("off,off_out,pad,pad_out", [(1, 1, 0, 0), (1, 0, 3, 8), (3, 3, 5, 5), (0, 7, 1, 2), (2, 5, 0, 16)])
def test_any_alignment_and_stride(dtype, off, off_out, pad, pad_out):
    """Rows that begin anywhere, the gradient's elsewhere; nothing beside them is written."""
    rows, V = 7, 4111
    x, vals, ids, lse, grad = make(6, rows, V, 30, dtype, rest=True)
    want = run(x, vals, ids, lse, 1.0, grad)

    def place(t, off, ld, fill):
        flat = torch.full((off + rows * ld + 8,), fill, dtype=DT[dtype], device="cuda")
        view = flat[off:off + rows * ld].view(rows, ld)[:, :V]
        if t is not None:
            view.copy_(t)
        return flat, view
    _, moved = place(x, off, V + pad, NAN)
    flat, out = place(None, off_out, V + pad_out, 44.0)
    loss, _ = run(moved, vals, ids, lse, 1.0, grad, out)
    T_eps = torch.finfo(DT[dtype]).eps
    # (sums meet in another order: a rounding of the result, and 2^-20)
    assert torch.allclose(loss, want[0], rtol=2.0 ** -19, atol=1e-6)
    assert torch.allclose(out.double(), want[1].double(), rtol=T_eps + 2.0 ** -19, atol=1e-7)
    beside = torch.ones_like(flat, dtype=torch.bool)
    beside[off_out:off_out + rows * (V + pad_out)].view(rows, -1)[:, :V] = False
    assert (flat[beside] == 44.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", [(3, 999), (5, 151_936), (400, 30_000)])
def test_in_place(dtype, rows, V):
    x, vals, ids, lse, grad = make(7, rows, V, 50, dtype, pad=3, rest=True)
    want = run(x, vals, ids, lse, 1.0, grad, torch.empty(rows, V + 3, dtype=x.dtype, device="cuda")[:, :V])
    got = run(x, vals, ids, lse, 1.0, grad, x)
    assert torch.equal(got[0], want[0]) and torch.equal(x, want[1])


def test_uint32_ids_and_no_loss():
    x, vals, ids, _, grad = make(8, 5, 700, 9, "f32")
    loss, out = run(x, vals, ids, None, 1.0, grad)
    a, b = run(x, vals, ids.view(torch.uint32), None, 1.0, grad)
    assert torch.equal(a, loss) and torch.equal(b, out)
    none, c = run(x, vals, ids, None, 1.0, grad, loss=False)
    assert none is None and torch.equal(c, out)


def test_no_rows():
    e = torch.empty(0, device="cuda")
    v, i = torch.empty(0, 4, device="cuda"), torch.empty(0, 4, dtype=torch.int32, device="cuda")
    B.sel_distill(torch.empty(0, 10, device="cuda"), v, i, None, 1.0, e)
    B.sel_distill_grad(torch.empty(0, 10, device="cuda"), v, i, e, 1.0, e, e, torch.empty(0, 10, device="cuda"))


@pytest.mark.parametrize("rows,V,dtype", [(6, 248_320, "f32"), (500, 30_001, "bf16")])
def test_results_do_not_depend_on_the_run(rows, V, dtype):
    x, vals, ids, lse, grad = make(9, rows, V, 100, dtype, rest=True)
    loss, out = run(x, vals, ids, lse, 1.0, grad)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            other = run(x, vals, ids, lse, 1.0, grad, stream=side)
        again = run(x, vals, ids, lse, 1.0, grad)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again + other, (loss, out) * 2))


@pytest.mark.parametrize("rest", [False, True])
def test_gradient_is_the_losses_differences(rest):
    rows, V, T = 12, 50, 2.0
    x, vals, ids, lse, grad = make(10, rows, V, 6, "f32", T, rest=rest)
    x = (x * 64).round() / 64  # (steps of 2^-5 are exact)
    _, out = run(x, vals, ids, lse, T, grad)
    h = 2.0 ** -5
    for j in list(range(0, V, 7)) + ids[:, 0].tolist()[:3]:
        e = torch.zeros(V, device="cuda")
        e[j] = h
        diff = (run(x + e, vals, ids, lse, T).double() - run(x - e, vals, ids, lse, T).double()) / (2 * h) * grad.double()
        # third derivatives of ln-sum-exps along one logit: below 0.1 / T^3 each, of two of
        # them with the rest; losses of about 2, off by 2^-20 of that
        tol = grad.double() * (2 * 0.1 / T ** 3 * h ** 2 / 6 + 2.0 ** -18 / h)
        assert ((diff - out[:, j].double()).abs() <= tol).all()


def test_offsets_past_32_bits():
    """Rows 2^31 entries apart: each its own."""
    rows, V, ld = 3, 5000, (1 << 31) + 8
    x, vals, ids, lse, grad = make(11, rows, V, 20, "bf16", rest=True)
    flat = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    view = flat.as_strided((rows, V), (ld, 1))
    view.copy_(x)
    want = run(x.contiguous(), vals, ids, lse, 1.0, grad)
    got = run(view, vals, ids, lse, 1.0, grad, view)
    assert torch.equal(got[0], want[0]) and torch.equal(view, want[1])
