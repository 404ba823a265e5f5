"""sel_head_w4 on the GPU against the 64-bit product."""
import numpy as np
import pytest
import torch

from oracle import decode as D
from sampling_row_fp32_gb300 import binding as B

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def make(seed, rows, V, H, group, zeros, dtype):
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 256, size=(V, H // 2), dtype=np.uint8)
    s = torch.from_numpy(rng.uniform(-0.02, 0.04, size=(V, H // group))).to(DT[dtype])
    z = torch.from_numpy(rng.integers(0, 256 if zeros == "any" else 16, size=(V, H // group), dtype=np.uint8)) if zeros else None
    x = torch.from_numpy(rng.normal(0, 1, size=(rows, H))).to(DT[dtype])
    return x, torch.from_numpy(q), s, z


def tolerance(mag, want, group, H, out):
    """Products are exact in fp32. A logit is a sum of `group` products a
    group, scaled, over H / group groups: at most group + H / group + 2
    roundings lie on a term's way, each at most a whole fp32 step (2^-23, as a
    truncating accumulator gives) of a sum no larger than the terms'
    magnitudes; then one rounding to the output type."""
    acc = (group + H // group + 2) * 2.0 ** -23 * mag + 2.0 ** -126  # (fp32's smallest normal)
    eps = torch.finfo(DT[out]).eps / 2
    return acc + eps * (np.abs(want) + acc) + torch.finfo(DT[out]).smallest_normal * eps


def check(x, q, s, z, group, out="f32", ld=None):
    rows, V, H = x.shape[0], q.shape[0], x.shape[1]
    ld = ld or V
    buf = torch.full((max(rows, 1), ld), -77.0, dtype=DT[out], device="cuda")
    logits = buf[:rows, :V]
    B.sel_head_w4(x.cuda(), q.cuda(), s.cuda(), None if z is None else z.cuda(), group, logits)
    want, mag = D.head_w4(x.double().numpy(), q.numpy(), s.double().numpy(), None if z is None else z.numpy(), group)
    got = logits.double().cpu().numpy()
    tol = tolerance(mag, want, group, H, out)
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol)
    assert (buf[:, V:] == -77.0).all()  # what lies between the rows is left as it was
    return logits


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,V,groups_per_row,zeros", [
    (1, 1, 1, None), (1, 300, 5, None), (2, 129, 3, "any"), (8, 128, 8, "nibble"), (9, 257, 7, None),
    (16, 1000, 2, "nibble"), (17, 513, 9, "any"), (33, 640, 4, None), (49, 1031, 11, "nibble"), (64, 256, 16, None),
    (65, 300, 3, "any"), (130, 77, 6, None)])
def test_shapes(dtype, group, rows, V, groups_per_row, zeros):
    check(*make(rows + V, rows, V, groups_per_row * group, group, zeros, dtype), group)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("ld", [None, 1035, 1040])
def test_output_types_and_strides(out, ld):
    check(*make(3, 5, 1031, 512, 64, "nibble", "bf16"), 64, out, ld)


@pytest.mark.parametrize("rows,V,H,group", [(8, 30_011, 8192, 64), (16, 30_011, 4096, 32), (13, 20_011, 4096, 128),
                                            (1, 20_011, 4096, 128), (49, 20_011, 4096, 64), (64, 9_999, 8192, 32), (7, 40_000, 2880, 32)])
def test_model_widths(rows, V, H, group):
    check(*make(rows, rows, V, H, group, None, "bf16"), group)


def test_every_nibble_at_every_place():
    """Weights one column at a time: column k's nibble of row v alone gets through."""
    H, V = 256, 512
    q = np.zeros((V, H // 2), dtype=np.uint8)
    for v in range(V):
        k = v % H
        q[v, k // 2] = (v % 16) << (4 * (k % 2))
    x = torch.arange(1, H + 1).to(torch.float16)[None]  # whole numbers up to 256: exact everywhere
    z = torch.zeros(V, H // 64, dtype=torch.uint8)
    s = torch.ones(V, H // 64, dtype=torch.float16)
    logits = check(x, torch.from_numpy(q), s, z, 64)
    want = torch.tensor([(v % 16) * (v % H + 1) for v in range(V)], dtype=torch.float32)
    assert torch.equal(logits[0].cpu(), want)


@pytest.mark.parametrize("rows", [1, 5, 12])
@pytest.mark.parametrize("low", [1e-3, 1e-9, 1e-30, 1e-40])
def test_hidden_states_of_a_wide_range(rows, low):
    """Values from `low` to 1e30 in one row, most of the weights of the large
    ones zero, so that the small ones decide: nothing of them may get lost."""
    x, q, s, z = make(rows, rows, 700, 512, 64, None, "bf16")
    rng = np.random.default_rng(1)
    big = torch.from_numpy(rng.random(x.shape) < 0.05)
    x = torch.where(big, x.float() * 1e30, x.float() * low).bfloat16()
    cols = big.any(0).numpy().nonzero()[0]
    qn = q.numpy()
    for k in cols:  # nibble 8: weight 0
        qn[:600, k // 2] = (qn[:600, k // 2] & (0xF0 if k % 2 == 0 else 0x0F)) | (8 << (4 * (k % 2)))
    check(x, q, s, z, 64)


@pytest.mark.parametrize("scale", [2.0 ** -130, 2.0 ** -100, 2.0 ** 100, 2.0 ** 122])
def test_hidden_states_at_the_ends_of_bf16(scale):
    x, q, s, z = make(2, 3, 300, 256, 128, "nibble", "bf16")
    x[1] = 0
    check((x.double() * scale).bfloat16(), q, s, z, 128)


@pytest.mark.parametrize("rows", [1, 6, 20])
@pytest.mark.parametrize("hidden,scale", [(2.0 ** -110, 2.0 ** 120), (2.0 ** 100, 2.0 ** -122), (2.0 ** 100, 2.0 ** -40)])
def test_small_hidden_states_meet_large_scales(rows, hidden, scale):
    """Only their products need to be in range, not a row's scaled sums."""
    x, q, s, z = make(11, rows, 300, 512, 64, "nibble", "bf16")
    check(x * hidden, q, s * scale, z, 64)


def test_no_rows():
    x, q, s, z = make(0, 0, 10, 64, 64, None, "bf16")
    B.sel_head_w4(x.cuda(), q.cuda(), s.cuda(), None, 64, torch.empty(0, 10, device="cuda"))


@pytest.mark.parametrize("rows", [3, 20, 40])
def test_nonfinite_inputs_fail_closed(rows):
    """A NaN hidden state or scale reaches its row's or column's logits and no others."""
    x, q, s, z = make(1, rows, 200, 256, 64, None, "bf16")
    x[1, 130] = float("nan")
    s[77, 2] = float("inf")
    logits = torch.empty(rows, 200, device="cuda")
    B.sel_head_w4(x.cuda(), q.cuda(), s.cuda(), None, 64, logits)
    finite = torch.isfinite(logits).cpu()
    want = torch.ones(rows, 200, dtype=torch.bool)
    want[1] = False
    want[:, 77] = False
    assert torch.equal(finite, want)


@pytest.mark.parametrize("rows", [2, 30, 70])
def test_results_do_not_depend_on_the_run(rows):
    """The same bits in every run, and with other work on a second stream."""
    x, q, s, z = (None if t is None else t.cuda() for t in make(5, rows, 5001, 1024, 32, "nibble", "f16"))
    outs = [torch.empty(rows, 5001, device="cuda") for _ in range(6)]
    other = torch.empty(rows, 5001, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for o in outs:
        with torch.cuda.stream(side):
            B.sel_head_w4(x, q, s, None, 32, other, side)
        B.sel_head_w4(x, q, s, z, 32, o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("rows", [4, 33])
@pytest.mark.parametrize("off", [2, 4, 6])
def test_entries_at_any_alignment(rows, off):
    """Scales `off` bytes and zero points off / 2 bytes past a 16-byte boundary."""
    x, q, s, z = make(6, rows, 999, 1024, 64, "nibble", "bf16")
    fs = torch.empty(s.numel() + 8, dtype=s.dtype, device="cuda")[off // 2:off // 2 + s.numel()].view(s.shape)
    fz = torch.empty(z.numel() + 16, dtype=z.dtype, device="cuda")[off // 2:off // 2 + z.numel()].view(z.shape)
    fs.copy_(s)
    fz.copy_(z)
    out, want = (torch.empty(rows, 999, device="cuda") for _ in range(2))
    B.sel_head_w4(x.cuda(), q.cuda(), fs, fz, 64, out)
    B.sel_head_w4(x.cuda(), q.cuda(), s.cuda(), z.cuda(), 64, want)
    assert torch.equal(out, want)


def test_offsets_past_32_bits():
    """A packed matrix of more than 2^32 bytes: its last rows are its own."""
    V, H = 1_060_000, 8192
    x, q, s, z = make(2, 2, 300, H, 128, None, "bf16")
    big_q = torch.zeros(V, H // 2, dtype=torch.uint8, device="cuda")
    big_s = torch.zeros(V, H // 128, dtype=torch.bfloat16, device="cuda")
    big_q[-300:], big_s[-300:] = q.cuda(), s.cuda()
    logits = torch.full((2, V), 5.0, device="cuda")
    B.sel_head_w4(x.cuda(), big_q, big_s, None, 128, logits)
    want, mag = D.head_w4(x.double().numpy(), q.numpy(), s.double().numpy(), None, 128)
    assert (np.abs(logits[:, -300:].double().cpu().numpy() - want) <= tolerance(mag, want, 128, H, "f32")).all()
    assert not logits[:, :-300].any()
