"""Argument checks of the operators around selection, and their plain forms
against hand-worked values (no GPU needed)."""
import ctypes
import os
import shutil

import numpy as np
import pytest
import torch

from oracle import decode as D

needs_nvcc = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc is needed to build the library")


@pytest.fixture(scope="module")
def lib():
    from sampling_row_fp32_gb300 import binding, build
    build.build()
    return binding.load()


@needs_nvcc
def test_head_validation(lib):
    from sampling_row_fp32_gb300 import binding as B
    vp, ok = ctypes.c_void_p, dict(x=0x10000, rows=3, q=0x10000, s=0x10000, z=None, group=64, dt=B.SEL_BF16, V=100,
                                   H=128, out=0x10000, odt=B.SEL_F32, ld=100)

    def head(**kw):
        a = {**ok, **kw}
        return lib.sel_head_w4(vp(a["x"]), a["rows"], vp(a["q"]), vp(a["s"]), vp(a["z"]), a["group"], a["dt"], a["V"],
                               a["H"], vp(a["out"]), a["odt"], a["ld"], None)
    assert head(rows=0, x=None, q=None, s=None, out=None) == B.SEL_OK
    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(out=None), dict(x=0x10008), dict(q=0x10008),
               dict(s=0x10001), dict(out=0x10002), dict(V=0), dict(V=0x80000000, ld=1 << 33), dict(H=0), dict(H=96),
               dict(H=(1 << 20) + 64), dict(dt=B.SEL_F32), dict(dt=7), dict(odt=3), dict(odt=-1), dict(ld=99),
               dict(ld=(1 << 40) + 1)):
        assert head(**kw) == B.SEL_EINVAL, kw
    for g in (0, 16, 48, 256):
        assert head(group=g, H=768) == B.SEL_EUNSUPPORTED


@needs_nvcc
def test_sample16_validation(lib):
    from sampling_row_fp32_gb300 import binding as B
    vp, f = ctypes.c_void_p, 0x10000
    ok = dict(x=f, dt=B.SEL_F16, rows=2, V=100, ld=100, T=f, k=f, p=f, m=f, u=f, ids=f, probs=f)

    def sample(**kw):
        a = {**ok, **kw}
        return lib.sel_sample16(vp(a["x"]), a["dt"], a["rows"], a["V"], a["ld"], *(vp(a[n]) for n in
                                ("T", "k", "p", "m", "u", "ids", "probs")), None)
    assert sample(rows=0, x=None, u=None, ids=None, probs=None) == B.SEL_OK
    for kw in (dict(x=None), dict(u=None), dict(ids=None), dict(probs=None), dict(x=f + 1), dict(T=f + 2), dict(k=f + 2),
               dict(p=f + 2), dict(m=f + 1), dict(u=f + 2), dict(ids=f + 2), dict(probs=f + 2), dict(V=0), dict(ld=99),
               dict(ld=(1 << 40) + 1), dict(dt=3), dict(dt=-1), dict(V=0x80000000, ld=1 << 33)):
        assert sample(**kw) == B.SEL_EINVAL, kw
    assert sample(dt=B.SEL_F32) == B.SEL_EUNSUPPORTED
    assert sample(V=B.SEL_SAMPLE16_MAX_V + 1, ld=1 << 20) == B.SEL_EUNSUPPORTED


@needs_nvcc
def test_embed_validation(lib):
    from sampling_row_fp32_gb300 import binding as B
    vp, f = ctypes.c_void_p, 0x10000

    def embed(ids=f, n=3, table=f, dt=B.SEL_F32, V=10, H=5, out=f):
        return lib.sel_embed(vp(ids), n, vp(table), dt, V, H, 1.0, vp(out), None)
    assert embed(n=0, ids=None, table=None, out=None) == B.SEL_OK
    for kw in (dict(ids=None), dict(table=None), dict(out=None), dict(ids=f + 2), dict(table=f + 2), dict(out=f + 2),
               dict(dt=3), dict(V=0), dict(H=0), dict(H=(1 << 20) + 1), dict(dt=B.SEL_F16, table=f + 1)):
        assert embed(**kw) == B.SEL_EINVAL, kw

    def w4(ids=f, n=3, q=f, s=f, z=None, group=32, dt=B.SEL_F16, V=10, H=64, out=f):
        return lib.sel_embed_w4(vp(ids), n, vp(q), vp(s), vp(z), group, dt, V, H, 1.0, vp(out), None)
    assert w4(n=0, ids=None, q=None, s=None, out=None) == B.SEL_OK
    for kw in (dict(ids=None), dict(q=None), dict(s=None), dict(out=None), dict(q=f + 8), dict(out=f + 8), dict(s=f + 1),
               dict(ids=f + 1), dict(dt=B.SEL_F32), dict(H=80), dict(H=0), dict(V=0)):
        assert w4(**kw) == B.SEL_EINVAL, kw
    assert w4(group=16) == B.SEL_EUNSUPPORTED


def test_binding_refuses_tensors_off_the_gpu():
    from sampling_row_fp32_gb300 import binding as B
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(5, 32, dtype=torch.uint8), torch.zeros(5, 1, dtype=torch.bfloat16)
    f, i = torch.zeros(2), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.sel_head_w4(x, q, s, None, 64, torch.zeros(2, 5))
    with pytest.raises(ValueError):
        B.sel_sample16(x, f, i, f, f, f, i, f)
    with pytest.raises(ValueError):
        B.sel_embed(i, torch.zeros(5, 64), 1.0, torch.zeros(2, 64))
    with pytest.raises(ValueError):
        B.sel_embed_w4(i, q, s, None, 64, 1.0, x)


def test_plain_dequantise_by_hand():
    q = np.array([[0x21, 0xF0]], dtype=np.uint8)  # columns 1, 2, 0, 15
    got = D.dequantise(q, np.array([[2.0, -0.5]]), np.array([[3, 15]], dtype=np.uint8), 2)
    assert got.tolist() == [[-4.0, -2.0, 7.5, 0.0]]
    assert D.dequantise(q, np.array([[1.0, 1.0]]), None, 2).tolist() == [[-7.0, -6.0, -8.0, 7.0]]


def test_plain_sample_by_hand():
    """Weights 1, 1/2, 1/2, 1/4 at T = 1 in the order ids 2, 0, 3, 1."""
    x = np.log(np.array([0.5, 0.25, 1.0, 0.5]))
    row = lambda k, p, m, u: D.sample16_row(x, 1.0, k, p, m, u)[0]  # noqa: E731
    assert [row(0, 1, 0, u) for u in (0.0, 0.43, 0.45, 0.66, 0.67, 0.88, 0.89)] == [2, 2, 0, 0, 3, 3, 1]
    assert [row(2, 1, 0, u) for u in (0.66, 0.67, 0.99)] == [2, 0, 0]
    assert [row(0, 0.5, 0, u) for u in (0.66, 0.67)] == [2, 0]   # 1 / 2.25 < 0.5: two ids
    assert [row(0, 0.44, 0, u) for u in (0.2, 0.99)] == [2, 2]   # 1 / 2.25 = 0.444
    assert [row(0, 1, 0.4, u) for u in (0.49, 0.51, 0.99)] == [2, 0, 3]
    assert D.sample16_row(x, 0.0, 3, 0.5, 0.1, 0.99) == (2, 1.0)
    assert D.sample16_row(np.array([1.0, 1.0, -np.inf]), 0.0, 0, 1, 0, 0.5) == (0, 1.0)
    assert D.sample16_row(np.array([-np.inf, -np.inf]), 1.0, 0, 1, 0, 0.5)[0] == D.INVALID
    assert D.sample16_row_exact(np.array([-np.inf, 1.0, 1.0, 1.0, 1.0]), 0, 0.5, 0.5) == (2, 0.5)
