"""The 4-bit head's tensor-core kernel on the GPU: matrices past 32 bits, entries
at any alignment in rows of odd lengths, and calls beside one another."""
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


def make(seed, rows, V, H, group, dtype):
    rng = np.random.default_rng(seed)
    q = torch.from_numpy(rng.integers(0, 256, size=(V, H // 2), dtype=np.uint8))
    s = torch.from_numpy(rng.uniform(-0.02, 0.04, size=(V, H // group))).to(dtype)
    z = torch.from_numpy(rng.integers(0, 16, size=(V, H // group), dtype=np.uint8))
    x = torch.from_numpy(rng.normal(0, 1, size=(rows, H))).to(dtype)
    return x, q, s, z


def near(got, x, q, s, z, group):
    """At most group + H / group + 2 roundings of a whole fp32 step lie on a term's
    way, each of a sum no larger than the terms' magnitudes."""
    want, mag = D.head_w4(x.double().numpy(), q.numpy(), s.double().numpy(), None if z is None else z.numpy(), group)
    off = np.abs(got.double().cpu().numpy() - want)
    return (off <= (group + x.shape[1] // group + 2) * 2.0 ** -23 * mag + 2.0 ** -126).all()


@pytest.mark.parametrize("rows", [20, 64])
def test_offsets_past_32_bits(rows):
    """A packed matrix of more than 2^32 bytes, and at 64 rows logits of more than
    2^32 / 4 elements behind a wide stride: the last rows are their own."""
    V, H, n = 1_060_000, 8192, 300
    x, q, s, z = make(2, rows, n, H, 128, torch.bfloat16)
    big_q = torch.zeros(V, H // 2, dtype=torch.uint8, device="cuda")
    big_s = torch.zeros(V, H // 128, dtype=torch.bfloat16, device="cuda")
    big_z = torch.zeros(V, H // 128, dtype=torch.uint8, device="cuda")
    big_q[-n:], big_s[-n:], big_z[-n:] = q.cuda(), s.cuda(), z.cuda()
    ld = V if rows < 64 else 70_000_000  # 64 rows: 4.48e9 elements
    buf = torch.empty((rows - 1) * ld + V, device="cuda")
    logits = torch.as_strided(buf, (rows, V), (ld, 1))
    logits.fill_(5.0)
    B.sel_head_w4(x.cuda(), big_q, big_s, big_z, 128, logits)
    assert near(logits[:, -n:], x, q, s, z, 128)
    assert not logits[:, :-n].any()


@pytest.mark.parametrize("rows", [5, 20, 49])
@pytest.mark.parametrize("off", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_entries_of_odd_rows_at_any_alignment(rows, off, dtype):
    """Groups of 32 in rows of 2,880 columns: 90 scales and 90 zero points a row,
    copied in narrow words, `off` entries past a 16-byte boundary."""
    V, H, group = 777, 2880, 32
    x, q, s, z = make(rows + off, rows, V, H, group, dtype)
    fs = torch.empty(s.numel() + 8, dtype=dtype, device="cuda")[off:off + s.numel()].view(s.shape)
    fz = torch.empty(z.numel() + 8, dtype=torch.uint8, device="cuda")[off:off + z.numel()].view(z.shape)
    fs.copy_(s)
    fz.copy_(z)
    logits = torch.empty(rows, V, device="cuda")
    B.sel_head_w4(x.cuda(), q.cuda(), fs, fz, group, logits)
    assert near(logits, x, q, s, z, group)


@pytest.mark.parametrize("rows", [2, 30, 70])
def test_two_streams_at_once(rows):
    """Each call's logits have the bits of the call alone, on both streams."""
    V, H, group = 5001, 1024, 32
    x, q, s, z = (t.cuda() for t in make(5, rows, V, H, group, torch.float16))
    alone, alone_z = (torch.empty(rows, V, device="cuda") for _ in range(2))
    B.sel_head_w4(x, q, s, None, group, alone)
    torch.cuda.synchronize()
    B.sel_head_w4(x, q, s, z, group, alone_z)
    torch.cuda.synchronize()
    outs, outs_z = ([torch.empty(rows, V, device="cuda") for _ in range(12)] for _ in range(2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for o, oz in zip(outs, outs_z):
        B.sel_head_w4(x, q, s, None, group, o, side)
        B.sel_head_w4(x, q, s, z, group, oz)
    torch.cuda.synchronize()
    assert all(torch.equal(o, alone) for o in outs)
    assert all(torch.equal(o, alone_z) for o in outs_z)
