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
