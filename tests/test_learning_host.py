"""The operators that a drafter learns with, without a GPU: the 64-bit forms that
the GPU tests compare with (against autograd and differences), the library's
checks of its arguments, and the binding's refusals."""
import ctypes
import itertools
import os
import shutil

import pytest
import torch

from oracle import learning as L
from sampling_row_fp32_gb300 import binding as B

needs_nvcc = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc is needed to build the library")
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    from sampling_row_fp32_gb300 import build
    build.build()
    return B.load()


# ---------------------------------------------------------------------------
# the 64-bit forms
# ---------------------------------------------------------------------------

def head_inputs(seed, n=6, V=11, H=5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, H, generator=g, dtype=torch.float64)
    w = torch.randn(V, H, generator=g, dtype=torch.float64)
    t = torch.randint(0, V, (n,), generator=g)
    t[2], t[4] = -1, V + 3
    return x, w, t, torch.rand(n, generator=g, dtype=torch.float64)


def test_head_loss_is_cross_entropy():
    x, w, t, _ = head_inputs(1)
    loss, lse = L.head_loss(x, w, t)
    live = [0, 1, 3, 5]
    want = torch.nn.functional.cross_entropy((x @ w.T)[live], t[live], reduction="none")
    assert torch.allclose(loss[live], want, rtol=1e-13) and not loss[[2, 4]].any()
    assert torch.allclose(lse, torch.logsumexp(x @ w.T, 1), rtol=1e-14)


def test_head_loss_near_zero_keeps_its_bits():
    """Two ids, the target 40 ahead: the loss is ln(1 + e^-40) = e^-40."""
    loss, _ = L.head_loss(torch.ones(1, 1, dtype=torch.float64), torch.tensor([[40.0], [0.0]]), torch.tensor([0]))
    assert abs(loss.item() / 4.248354255291589e-18 - 1) < 1e-12


def test_head_loss_grad_is_autograds():
    x, w, t, g = head_inputs(2)
    x.requires_grad_()
    w.requires_grad_()
    loss, lse = L.head_loss(x, w, t)
    (loss * g).sum().backward()
    dx, dw = L.head_loss_grad(x.detach(), w.detach(), t, lse.detach(), g)
    assert torch.allclose(dx, x.grad, rtol=1e-12, atol=1e-14) and torch.allclose(dw, w.grad, rtol=1e-12, atol=1e-14)


def test_head_loss_grad_is_the_differences():
    x, w, t, g = head_inputs(3)
    _, lse = L.head_loss(x, w, t)
    dx, dw = L.head_loss_grad(x, w, t, lse, g)
    h = 1e-5
    f = lambda a, b: (L.head_loss(a, b, t)[0] * g).sum().item()  # noqa: E731
    for p, d in ((x, dx), (w, dw)):
        for i in range(0, p.numel(), 7):
            e = torch.zeros_like(p).view(-1)
            e[i] = h
            e = e.view(p.shape)
            up, down = (f(x + e, w), f(x - e, w)) if p is x else (f(x, w + e), f(x, w - e))
            assert abs((up - down) / (2 * h) - d.reshape(-1)[i].item()) < 1e-9


def lists(seed, n=5, V=13, k=4):
    g = torch.Generator().manual_seed(seed)
    teacher = 2 * torch.randn(n, V, generator=g, dtype=torch.float64)
    x = torch.randn(n, V, generator=g, dtype=torch.float64)
    vals, ids = torch.topk(teacher, k, dim=1)
    return teacher, x, vals, ids, torch.rand(n, generator=g, dtype=torch.float64)


def test_distill_over_a_whole_vocabulary_is_the_divergence():
    teacher, x, _, _, _ = lists(1)
    T = 1.5
    vals, ids = torch.topk(teacher, 13, dim=1)
    p, q = torch.softmax(teacher / T, 1), torch.softmax(x / T, 1)
    want = (p * (p / q).log()).sum(1)
    assert torch.allclose(L.distill(x, vals, ids, None, T), want, rtol=1e-12)
    assert torch.allclose(L.distill(x, vals, ids, torch.logsumexp(teacher / T, 1), T), want, rtol=1e-12)


@pytest.mark.parametrize("rest", [False, True])
def test_distill_grad_is_autograds_and_the_differences(rest):
    teacher, x, vals, ids, g = lists(2)
    T = 0.75
    ids[1, 2:] = -1
    lse = torch.logsumexp(teacher / T, 1) if rest else None
    loss, grad = L.distill(x, vals, ids, lse, T, g)
    x.requires_grad_()
    total = 0
    for r in range(len(x)):
        e = ids[r] >= 0
        lp = vals[r, e] / T - (lse[r] if rest else torch.logsumexp(vals[r, e] / T, 0))
        lq = torch.log_softmax(x[r] / T, 0)
        one = (lp.exp() * (lp - lq[ids[r, e]])).sum()
        if rest:
            left, others = 1 - lp.exp().sum(), 1 - lq[ids[r, e]].exp().sum()
            one = one + left * (left / others).log()
        assert torch.allclose(loss[r], one.detach(), rtol=1e-11)
        total = total + g[r] * one
    total.backward()
    assert torch.allclose(grad, x.grad, rtol=1e-10, atol=1e-14)
    x = x.detach()
    h = 1e-5
    for i in range(0, x.numel(), 5):
        e = torch.zeros_like(x).view(-1)
        e[i] = h
        e = e.view(x.shape)
        diff = ((L.distill(x + e, vals, ids, lse, T) - L.distill(x - e, vals, ids, lse, T)) * g).sum() / (2 * h)
        assert abs(diff.item() - grad.reshape(-1)[i].item()) < 1e-8


def test_distill_rows_that_do_not_count_or_fail():
    _, x, vals, ids, g = lists(3)
    ids[0] = -1
    vals[1] = -INF
    ids[2, 1] = ids[2, 0]
    x[3, 5] = NAN
    loss, grad = L.distill(x, vals, ids, None, 1.0, g)
    assert loss[0] == 0 and loss[1] == 0 and not grad[:2].any()
    assert torch.isnan(loss[2:4]).all() and torch.isnan(grad[2:4]).all()
    assert torch.isfinite(loss[4]) and torch.isfinite(grad[4]).all()


# ---------------------------------------------------------------------------
# the library's checks (no pointer is followed)
# ---------------------------------------------------------------------------

F = 0x10000
WS = 1 << 40


@needs_nvcc
def test_head_loss_validation(lib):
    vp = ctypes.c_void_p

    def loss(x=F, rows=3, w=F, dt=B.SEL_BF16, V=10, H=16, t=F, out=F, lse=F, ws=F, n=WS):
        return lib.sel_head_loss(vp(x), rows, vp(w), dt, V, H, vp(t), vp(out), vp(lse), vp(ws), n, None)
    assert loss(rows=0, x=None, w=None, t=None, out=None, lse=None, ws=None, n=0) == B.SEL_OK
    for kw in (dict(x=None), dict(w=None), dict(t=None), dict(out=None), dict(ws=None), dict(x=F + 8), dict(w=F + 8),
               dict(t=F + 2), dict(out=F + 2), dict(lse=F + 1), dict(ws=F + 128), dict(dt=B.SEL_F32), dict(dt=7),
               dict(V=0), dict(V=0x80000000), dict(H=0), dict(H=(1 << 20) + 8)):
        assert loss(**kw) == B.SEL_EINVAL, kw
    assert loss(H=12) == B.SEL_EUNSUPPORTED
    assert loss(rows=0x80000000) == B.SEL_EUNSUPPORTED
    assert loss(rows=0x7fffffff, V=0x7fffffff) == B.SEL_EUNSUPPORTED
    need = B.sel_workspace_bytes(B.SEL_OP_HEAD_LOSS, 3, 10, 16)
    assert need > 0 and loss(n=need - 1) == B.SEL_EWORKSPACE


@needs_nvcc
def test_head_loss_grad_validation(lib):
    vp = ctypes.c_void_p

    def grad(x=F, rows=3, w=F, dt=B.SEL_F16, V=10, H=16, t=F, lse=F, g=F, dx=F, dw=F, ws=F, n=WS):
        return lib.sel_head_loss_grad(vp(x), rows, vp(w), dt, V, H, vp(t), vp(lse), vp(g), vp(dx), vp(dw), vp(ws), n, None)
    assert grad(rows=0, x=None, w=None, t=None, lse=None, g=None, dw=None, ws=None, n=0) == B.SEL_OK
    for kw in (dict(x=None), dict(w=None), dict(t=None), dict(lse=None), dict(g=None), dict(dx=None, dw=None), dict(ws=None),
               dict(dx=F + 8), dict(dw=F + 8), dict(lse=F + 2), dict(g=F + 2), dict(ws=F + 64), dict(dt=B.SEL_F32),
               dict(V=0), dict(H=0)):
        assert grad(**kw) == B.SEL_EINVAL, kw
    assert grad(H=20) == B.SEL_EUNSUPPORTED
    need = B.sel_workspace_bytes(B.SEL_OP_HEAD_LOSS_GRAD, 3, 10, 16)
    assert need > 0 and grad(n=need - 1) == B.SEL_EWORKSPACE


@needs_nvcc
def test_workspaces(lib):
    for op in (B.SEL_OP_HEAD_LOSS, B.SEL_OP_HEAD_LOSS_GRAD):
        assert B.sel_workspace_bytes(op, 0, 10, 16) == 0
        assert B.sel_workspace_bytes(op, 3, 0, 16) == 0
        assert B.sel_workspace_bytes(op, 3, 10, 12) == 0
        assert B.sel_workspace_bytes(op, 3, 10, 0) == 0
        assert B.sel_workspace_bytes(op, 0x7fffffff, 0x7fffffff, 16) == 0
        # a larger call's workspace serves a smaller one
        sizes = [(1, 15, 16, 17, 100, 128, 129, 255, 256, 257, 300, 511, 777, 1024, 4096, 4097, 20_000, 300_000),
                 (1, 255, 256, 257, 16_384, 16_385, 93_001, 151_936, 248_320), (8, 248, 256, 264, 2880, 4096)]
        need = {k: B.sel_workspace_bytes(op, *k) for k in itertools.product(*sizes)}
        assert min(need.values()) > 0
        for k, n in need.items():
            for axis in range(3):
                at = sizes[axis].index(k[axis])
                if at:
                    assert need[k[:axis] + (sizes[axis][at - 1],) + k[axis + 1:]] <= n, (op, k, axis)
    # far below the logits it does not keep (4,096 x 151,936 in fp32: 2.5 GB)
    assert B.sel_workspace_bytes(B.SEL_OP_HEAD_LOSS, 4096, 151_936, 4096) < 64 << 20
    assert B.sel_workspace_bytes(B.SEL_OP_HEAD_LOSS_GRAD, 4096, 151_936, 4096) < 800 << 20


@needs_nvcc
def test_distill_validation(lib):
    vp = ctypes.c_void_p

    def distill(x=F, dt=B.SEL_F32, rows=3, V=10, ld=10, v=F, i=F, k=4, lse=F, T=1.0, loss=F):
        return lib.sel_distill(vp(x), dt, rows, V, ld, vp(v), vp(i), k, vp(lse), T, vp(loss), None)

    def grad(x=F, dt=B.SEL_F32, rows=3, V=10, ld=10, v=F, i=F, k=4, lse=F, T=1.0, g=F, loss=F, out=2 * F, ld_out=10):
        return lib.sel_distill_grad(vp(x), dt, rows, V, ld, vp(v), vp(i), k, vp(lse), T, vp(g), vp(loss), vp(out), ld_out,
                                    None)
    assert distill(rows=0, x=None, v=None, i=None, lse=None, loss=None) == B.SEL_OK
    assert grad(rows=0, x=None, v=None, i=None, lse=None, g=None, loss=None, out=None) == B.SEL_OK
    for f in (distill, grad):
        for kw in (dict(x=None), dict(v=None), dict(i=None), dict(x=F + 2), dict(v=F + 2), dict(i=F + 1), dict(lse=F + 2),
                   dict(loss=F + 2), dict(dt=3), dict(dt=-1), dict(V=0, k=1), dict(ld=9), dict(ld=(1 << 40) + 1), dict(k=0),
                   dict(k=11), dict(T=0.0), dict(T=-1.0), dict(T=INF), dict(T=NAN), dict(x=F + 1, dt=B.SEL_BF16)):
            assert f(**kw) == B.SEL_EINVAL, (f.__name__, kw)
        assert f(V=5000, ld=5000, k=1025, **({"ld_out": 5000} if f is grad else {})) == B.SEL_EUNSUPPORTED
        V = (1 << 20) + 1
        assert f(V=V, ld=V, **({"ld_out": V} if f is grad else {})) == B.SEL_EUNSUPPORTED
        assert f(rows=0x80000000) == B.SEL_EUNSUPPORTED
    assert distill(loss=None) == B.SEL_EINVAL
    for kw in (dict(g=None), dict(out=None), dict(g=F + 2), dict(out=F + 2), dict(ld_out=9), dict(out=F, ld=12, ld_out=10)):
        assert grad(**kw) == B.SEL_EINVAL, kw


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------

class Reached:
    def __getattr__(self, name):
        def call(*args):
            raise AssertionError(f"{name} was called")
        return call


@pytest.fixture
def no_gpu(monkeypatch):
    monkeypatch.setattr(B, "_device", lambda *tensors: 0)
    monkeypatch.setattr(B, "_on_stream", lambda stream, dev: 0)
    monkeypatch.setattr(B, "_lib", Reached())


def m(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


BIG = 2 ** 32 + 5
f32, i32 = torch.float32, torch.int32


def head_call(rows=4, V=9, H=16, x=None, w=None, t=None, loss=None, lse=None):
    B.sel_head_loss(m(rows, H) if x is None else x, m(V, H) if w is None else w, m(rows, dtype=i32) if t is None else t,
                    m(rows, dtype=f32) if loss is None else loss, m(rows, dtype=f32) if lse is None else lse, None)


def grad_call(rows=4, V=9, H=16, dx=None, dw=None, lse=None, g=None):
    B.sel_head_loss_grad(m(rows, H), m(V, H), m(rows, dtype=i32), m(rows, dtype=f32) if lse is None else lse,
                         m(rows, dtype=f32) if g is None else g, m(rows, H) if dx is None else dx,
                         m(V, H) if dw is None else dw, None)


def distill_call(rows=4, V=9, k=3, x=None, v=None, i=None, lse=None, g=None, loss=None, out=None):
    x = m(rows, V) if x is None else x
    v, i = m(rows, k, dtype=f32) if v is None else v, m(rows, k, dtype=i32) if i is None else i
    loss = m(rows, dtype=f32) if loss is None else loss
    if out is None and g is None:
        B.sel_distill(x, v, i, lse, 1.0, loss)
    else:
        B.sel_distill_grad(x, v, i, lse, 1.0, m(rows, dtype=f32) if g is None else g, loss, m(rows, V) if out is None else out)


@pytest.mark.parametrize("call", [
    lambda: head_call(rows=BIG),
    lambda: head_call(V=BIG),
    lambda: head_call(H=2 ** 32),
    lambda: head_call(w=m(9, 24)),
    lambda: head_call(w=m(9, 16, dtype=torch.float16)),
    lambda: head_call(x=m(4, 16, dtype=f32), w=m(9, 16, dtype=f32)),
    lambda: head_call(x=m(16, 4).t()),
    lambda: head_call(w=m(16, 9).t()),
    lambda: head_call(t=m(5, dtype=i32)),
    lambda: head_call(t=m(4, dtype=torch.int64)),
    lambda: head_call(loss=m(4)),
    lambda: head_call(lse=m(3, dtype=f32)),
    lambda: grad_call(dx=m(4, 16, dtype=f32)),
    lambda: grad_call(dx=m(4, 8)),
    lambda: grad_call(dw=m(16, 9).t()),
    lambda: grad_call(lse=m(4)),
    lambda: grad_call(g=m(4, 1, dtype=f32)),
    lambda: distill_call(rows=BIG, V=1, k=1),
    lambda: distill_call(V=BIG),
    lambda: distill_call(k=BIG),
    lambda: distill_call(x=m(4, 9, dtype=torch.float64)),
    lambda: distill_call(x=m(9, 4).t()),
    lambda: distill_call(v=m(4, 3)),
    lambda: distill_call(v=m(3, 3, dtype=f32)),
    lambda: distill_call(i=m(4, 2, dtype=i32)),
    lambda: distill_call(i=m(4, 3, dtype=torch.int64)),
    lambda: distill_call(v=m(4, 6, dtype=f32)[:, ::2]),
    lambda: distill_call(lse=m(5, dtype=f32)),
    lambda: distill_call(loss=m(4)),
    lambda: distill_call(g=m(3, dtype=f32)),
    lambda: distill_call(out=m(4, 9, dtype=f32)),
    lambda: distill_call(out=m(4, 8)),
])
def test_binding_refuses(no_gpu, call):
    with pytest.raises(ValueError):
        call()


def test_binding_lets_through(no_gpu):
    for call, name in ((head_call, "sel_head_loss"), (grad_call, "sel_head_loss_grad"), (distill_call, "sel_distill"),
                       (lambda: distill_call(out=m(4, 12)[:, :9]), "sel_distill_grad")):
        with pytest.raises(AssertionError, match=f"{name} was called"):
            call()


def test_binding_refuses_tensors_off_the_gpu():
    x, w, f, i = torch.zeros(2, 16).half(), torch.zeros(5, 16).half(), torch.zeros(2), torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError):
        B.sel_head_loss(x, w, i, f, f, None)
    with pytest.raises(ValueError):
        B.sel_head_loss_grad(x, w, i, f, f, x, w, None)
    with pytest.raises(ValueError):
        B.sel_distill(x, f[:, None], i[:, None], None, 1.0, f)
    with pytest.raises(ValueError):
        B.sel_distill_grad(x, f[:, None], i[:, None], None, 1.0, f, f, x)
