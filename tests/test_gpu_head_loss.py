"""sel_head_loss and sel_head_loss_grad on the GPU against the 64-bit formulas."""
import numpy as np
import pytest
import torch

from oracle import learning as L
from sampling_row_fp32_gb300 import binding as B

pytestmark = pytest.mark.gpu

NAN = float("nan")
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def make(seed, rows, V, H, dtype, spread=2.0, ignored=0.2):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(V, H, generator=g) * spread / H ** 0.5).to(DT[dtype])
    t = torch.randint(0, V, (rows,), generator=g)
    x = torch.randn(rows, H, generator=g)
    x[::2] += 4.0 * torch.rand((rows + 1) // 2, 1, generator=g) * w[t[::2]].float()  # rows that know their token
    t = torch.where(torch.rand(rows, generator=g) < ignored, -1, t)
    grad = (0.5 + torch.rand(rows, generator=g)) * (256.0 if dtype == "f16" else 1.0)
    return x.to(DT[dtype]).cuda(), w.cuda(), t.to(torch.int32).cuda(), grad.cuda()


def run_loss(x, w, t, stream=None, ws=None):
    rows, V, H = x.shape[0], w.shape[0], x.shape[1]
    ws = B.workspace(B.SEL_OP_HEAD_LOSS, rows, V, H) if ws is None else ws
    loss, lse = (torch.full((rows,), -77.0, device="cuda") for _ in range(2))
    B.sel_head_loss(x, w, t, loss, lse, ws, stream)
    return loss, lse


def run_grad(x, w, t, lse, grad, ws=None):
    rows, V, H = x.shape[0], w.shape[0], x.shape[1]
    ws = B.workspace(B.SEL_OP_HEAD_LOSS_GRAD, rows, V, H) if ws is None else ws
    dx, dw = torch.full_like(x, -77.0), torch.full_like(w, -77.0)
    B.sel_head_loss_grad(x, w, t, lse, grad, dx, dw, ws)
    assert int(ws[:4].view(torch.int32).item()) == 0
    return dx, dw


def logit_error(x, w):
    """Of each row, the most a logit may be off: products are exact in fp32, and at
    most H + 2 roundings lie on a term's way, each a whole fp32 step (2^-23, as a
    truncating accumulator gives) of a sum no larger than the terms' magnitudes."""
    mag = x.double().abs() @ w.double().abs().T
    return (x.shape[1] + 2) * 2.0 ** -23 * mag


def check_loss(x, w, t):
    loss, lse = run_loss(x, w, t)
    want, want_lse = L.head_loss(x, w, t)
    dz = logit_error(x, w).max(dim=1).values
    # The statistics: each weight has an exponent rounded to 2^-24 of itself (which
    # counts as it shrinks, at most 2^-23) and 2^-22 of the exponential; a sum of 32 in
    # four runs, over four chunks, adds 15 roundings, the joins are finer: below 2^-19.
    # A loss moves by 1 - exp(-loss) times what the difference of its logits does.
    d = 2 * dz + 2.0 ** -19
    tol = (1 - torch.exp(-want)) * d * (1 + d) + 2.0 ** -23 * want + 2.0 ** -126
    err = (loss.double() - want).abs()
    assert (err <= tol).all(), (err / tol).max()
    err = (lse.double() - want_lse).abs()
    tol = dz + 2.0 ** -19 + 2.0 ** -23 * want_lse.abs()
    assert (err <= tol).all(), (err / tol).max()
    return loss, lse


def check_grad(x, w, t, lse, grad):
    dx, dw = run_grad(x, w, t, lse, grad)
    want_x, want_w = L.head_loss_grad(x, w, t, lse, grad)
    T = x.dtype
    eps = torch.finfo(T).eps / 2
    V, rows = w.shape[0], x.shape[0]
    x64, w64, l64 = x.double(), w.double(), lse.double()
    tl = t.long()
    live = (tl >= 0) & (tl < V) & (grad != 0)
    p = torch.exp(x64 @ w64.T - l64[:, None])
    p[~live] = 0
    # An entry of P: its logit's error and that of the exponential (its exponent, z -
    # lse rounded, moves it by 2^-23 |z - lse|, and |d| e^d <= 1 below), the same on
    # the target's e^d - 1, whose own rounding and that to T come on top; f16 holds it
    # 2^14 up times at least 1/2, where 2^-25 is half its smallest step.
    dz = logit_error(x, w) + 2.0 ** -20
    depth = 1 + (x64 @ w64.T - l64[:, None]).abs()
    dp = p * (dz + 2.0 ** -23 * depth) * (1 + 2.0 ** -8)
    hot = torch.zeros_like(p)
    hot[live, tl[live]] = 1.0
    a = (p - hot).abs()
    dp = dp + a * (eps + 2.0 ** -22) + (2.0 ** -38 if T == torch.float16 else 2.0 ** -134) * live[:, None]
    g = grad.double().abs() * live
    # sums: a rounding of a whole fp32 step for each term, as above
    mag = (a + dp) @ w64.abs()
    tol = g[:, None] * (dp @ w64.abs() + (V + 300) * 2.0 ** -23 * mag)
    tiny = torch.finfo(T).smallest_normal * eps
    tol = tol + eps * (want_x.abs() + tol) + tiny
    err = (dx.double() - want_x).abs()
    assert (err <= tol).all(), (err / tol).max()
    assert not dx[~live].any()
    # hidden rows times a power of two: exact but for what becomes subnormal
    top = g.max()
    u = x64.abs()
    small = torch.where(live & (g < top), tiny * (1 + top / torch.where(live, g, 1.0)), 0.0)  # (dead rows: no 0 * inf)
    du = small[:, None].expand_as(u)
    ga, gd = a * g[:, None], dp * g[:, None]
    tol = gd.T @ u + ga.T @ du + gd.T @ du
    tol = tol + (rows + 4) * 2.0 ** -23 * ((ga + gd).T @ u)
    tol = tol + eps * (want_w.abs() + tol) + tiny
    err = (dw.double() - want_w).abs()
    assert (err <= tol).all(), (err / tol).max()
    return dx, dw


SHAPES = [(1, 1, 8), (1, 300, 64), (2, 129, 72), (31, 256, 128), (49, 1000, 264), (127, 257, 520), (128, 512, 64),
          (129, 513, 64), (200, 127, 136), (256, 1031, 512), (257, 2, 40), (300, 3001, 1000), (600, 700, 2880)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,V,H", SHAPES)
def test_loss(rows, V, H, dtype):
    x, w, t, _ = make(rows + V, rows, V, H, dtype)
    check_loss(x, w, t)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,V,H", SHAPES)
def test_grad(rows, V, H, dtype):
    x, w, t, grad = make(rows + V, rows, V, H, dtype)
    _, lse = run_loss(x, w, t)
    check_grad(x, w, t, lse, grad)


@pytest.mark.parametrize("rows,V,H", [(16_400, 17_000, 64), (1, 151_936, 256), (20, 60_001, 512), (300, 40_000, 72)])
def test_pieces_and_long_vocabularies(rows, V, H):
    x, w, t, grad = make(rows, rows, V, H, "bf16")
    _, lse = check_loss(x, w, t)
    check_grad(x, w, t, lse, grad)


def test_equal_gradients_round_hidden_rows_once():
    """A mean's gradients: hidden rows enter dW unrounded, and check_grad allows nothing for them."""
    x, w, t, _ = make(3, 200, 500, 64, "bf16")
    _, lse = run_loss(x, w, t)
    check_grad(x, w, t, lse, torch.full((200,), 1 / 160, device="cuda"))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gradients_of_both_signs_and_very_different_sizes(dtype):
    x, w, t, grad = make(4, 140, 300, 128, dtype)
    grad = grad * torch.where(torch.arange(140, device="cuda") % 3 == 0, -1.0, 1.0)
    grad = grad * 2.0 ** -(torch.arange(140, device="cuda") % 9)
    _, lse = run_loss(x, w, t)
    check_grad(x, w, t, lse, grad)


@pytest.mark.parametrize("rows", [5, 260])
def test_one_output_alone_is_the_same(rows):
    x, w, t, grad = make(5, rows, 700, 200, "bf16")
    _, lse = run_loss(x, w, t)
    dx, dw = run_grad(x, w, t, lse, grad)
    ws = B.workspace(B.SEL_OP_HEAD_LOSS_GRAD, rows, 700, 200)
    a, b = torch.full_like(x, 9.0), torch.full_like(w, 9.0)
    B.sel_head_loss_grad(x, w, t, lse, grad, a, None, ws)
    B.sel_head_loss_grad(x, w, t, lse, grad, None, b, ws)
    assert torch.equal(b, dw)
    # (dX's sums are split alike whether dW is there or not)
    assert torch.equal(a, dx)


@pytest.mark.parametrize("rows", [3, 200])
def test_rows_that_do_not_count_hold_anything(rows):
    x, w, t, grad = make(6, rows, 400, 96, "bf16", ignored=0.0)
    t[0], t[2] = -1, 400  # (the first id past the vocabulary)
    if rows > 100:
        t[100] = 0x7FFFFFFF
        grad[150] = 0.0
    x[0], grad[2] = NAN, NAN
    loss, lse = run_loss(x, w, t)
    assert not loss[[0, 2]].any() and torch.isfinite(loss).all() and torch.isnan(lse[0])
    dx, dw = run_grad(x, w, t, lse, grad)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all() and not dx[[0, 2]].any()
    clean = x.clone()
    clean[0] = 0
    g = torch.nan_to_num(grad)
    same = run_grad(clean, w, t, run_loss(clean, w, t)[1], g)
    assert torch.equal(dx, same[0]) and torch.equal(dw, same[1])


@pytest.mark.parametrize("rows", [2, 300])
def test_no_row_counts(rows):
    x, w, t, grad = make(7, rows, 300, 64, "f16")
    t.fill_(-1)
    loss, lse = run_loss(x, w, t)
    assert not loss.any() and torch.allclose(lse.double(), L.head_loss(x, w, t)[1], atol=1e-4)
    dx, dw = run_grad(x, w, t, lse, grad)
    assert not dx.any() and not dw.any()


@pytest.mark.parametrize("rows", [4, 260])
def test_nonfinite_values_reach_what_they_are_part_of(rows):
    x, w, t, grad = make(8, rows, 500, 64, "bf16", ignored=0.0)
    x[1, 3] = NAN
    x[2] = 0
    x[2, 5] = float("inf")  # infinities of both signs among its logits
    loss, lse = run_loss(x, w, t)
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[1:3] = True
    assert torch.equal(torch.isnan(loss), bad) and torch.equal(torch.isnan(lse), bad)
    dx, dw = run_grad(x, w, t, lse, grad)
    assert torch.isnan(dx[1:3]).all() and torch.isfinite(dx[~bad]).all() and torch.isnan(dw).all()
    # a weight of -Inf where the hidden row is positive: a logit of -Inf, a probability of 0
    x, w, t, grad = make(9, rows, 500, 64, "bf16", ignored=0.0)
    x[:, 7] = x[:, 7].abs() + 0.5
    w[77, 7] = -float("inf")
    t[0] = 77
    loss, lse = run_loss(x, w, t)
    assert loss[0] == float("inf") and torch.isfinite(loss[1:][t[1:] != 77]).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("rows", [1, 40, 256])
@pytest.mark.parametrize("scale", [2.0 ** 8, 2.0 ** 30, 2.0 ** 60])
def test_logits_of_any_size(rows, scale):
    """Logits so far apart that one id has all the weight: the loss is their difference."""
    x, w, t, _ = make(10, rows, 300, 64, "bf16", ignored=0.0)
    loss, lse = run_loss((x.double() * scale).to(x.dtype), w, t)
    z = x.double() @ w.double().T * scale
    want = torch.logsumexp(z, 1)
    tol = 2 * logit_error(x, w).max(dim=1).values * scale + 2.0 ** -19 + 2.0 ** -22 * want.abs()
    assert ((lse.double() - want).abs() <= tol).all()
    assert ((loss.double() - (want - z[torch.arange(rows), t.long()])).abs() <= 2 * tol).all()


def test_confident_rows_keep_the_bits_of_their_losses():
    """Losses down to 1e-30: relative precision, as the definition has it."""
    H, V = 64, 300
    w = torch.zeros(V, H, device="cuda", dtype=torch.bfloat16)
    w[:, 0] = torch.arange(V, device="cuda") % 2 * 0.125
    w[5, 0], w[5, 1] = 0, 1.0
    x = torch.zeros(70, H, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = 1.0
    x[:, 1] = torch.arange(70, device="cuda").bfloat16()  # the target's logit: whole numbers, exact
    t = torch.full((70,), 5, dtype=torch.int32, device="cuda")
    loss, _ = run_loss(x, w, t)
    want, _ = L.head_loss(x, w, t)
    assert want.min() < 1e-27
    assert ((loss.double() / want - 1).abs() < 2.0 ** -18).all()


@pytest.mark.parametrize("rows", [5, 90, 300])
def test_results_do_not_depend_on_the_run_or_the_workspace(rows):
    """The same bits from a workspace full of anything but its error word, and with
    other work on a second stream."""
    x, w, t, grad = make(11, rows, 5000, 264, "f16")
    loss, lse = run_loss(x, w, t)
    dx, dw = run_grad(x, w, t, lse, grad)
    side = torch.cuda.Stream()
    ws = [B.workspace(op, 400, 6000, 512) for op in (B.SEL_OP_HEAD_LOSS, B.SEL_OP_HEAD_LOSS_GRAD)]
    other = B.workspace(B.SEL_OP_HEAD_LOSS, rows, 5000, 264), torch.empty(rows, device="cuda")
    torch.cuda.synchronize()
    for fill in (0, 255, 127):
        for b in ws:
            b[4:].fill_(fill)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            B.sel_head_loss(x, w, t, other[1], None, other[0], side)
        again = run_loss(x, w, t, ws=ws[0])
        assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])
        again = run_grad(x, w, t, lse, grad, ws=ws[1])
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    assert torch.equal(other[1], loss)


def test_no_rows():
    x, w, t, grad = make(0, 0, 10, 64, "bf16")
    e = torch.empty(0, device="cuda")
    B.sel_head_loss(x, w, t, e, e, None)
    dw = torch.full_like(w, 5.0)
    B.sel_head_loss_grad(x, w, t, e, e, x, dw, None)
    assert not dw.any()


def test_uint32_targets_and_no_lse():
    x, w, t, _ = make(12, 33, 200, 64, "bf16")
    loss, _ = run_loss(x, w, t)
    got = torch.empty_like(loss)
    B.sel_head_loss(x, w, t.view(torch.uint32), got, None, B.workspace(B.SEL_OP_HEAD_LOSS, 33, 200, 64))
    assert torch.equal(got, loss)


def test_a_raised_error_word_fails_every_row():
    """What a wait that runs out does: here the word is raised by the host."""
    x, w, t, grad = make(13, 20, 300, 64, "bf16")
    lse = run_loss(x, w, t)[1]
    ws = B.workspace(B.SEL_OP_HEAD_LOSS_GRAD, 20, 300, 64)
    ws[0] = 1
    assert all(torch.isnan(o).all() for o in run_loss(x, w, t, ws=ws))
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    B.sel_head_loss_grad(x, w, t, lse, grad, dx, dw, ws)
    assert torch.isnan(dx).all() and torch.isnan(dw).all()


def test_gradient_is_the_losses_differences():
    """Central differences of the losses the kernel gives. Hidden states are whole
    multiples of 2^-5 below 4 and the step is 2^-4: exact in f16."""
    rows, V, H = 40, 200, 64
    _, w, t, grad = make(14, rows, V, H, "f16")
    grad = grad / 256
    x = (torch.randint(-100, 100, (rows, H), generator=torch.Generator().manual_seed(1)) / 32).half().cuda()
    _, lse = run_loss(x, w, t)
    dx, _ = check_grad(x, w, t, lse, grad)
    h = 2.0 ** -4
    for k in range(0, H, 9):
        e = torch.zeros(H, device="cuda", dtype=torch.float16)
        e[k] = h
        up, down = run_loss(x + e, w, t)[0].double(), run_loss(x - e, w, t)[0].double()
        # (a row's difference moves none of the others)
        diff = grad.double() * (up - down) / (2 * h)
        # the third derivative is w[:, k]'s third cumulant: below 0.1 of its range cubed;
        # the losses' own errors as in check_loss, the gradient's as in check_grad (2^-11 of
        # it and of P's terms, whose magnitudes sum to at most 2 max |w|)
        r = (w[:, k].double().max() - w[:, k].double().min()).item()
        dz = logit_error(x + e, w).max(dim=1).values
        tol = 0.1 * r ** 3 * h ** 2 / 6 + (2 * dz + 2.0 ** -19 + 2.0 ** -23 * up.abs().max()) / h
        tol = grad.double() * (tol + 2.0 ** -10 * 3 * w[:, k].double().abs().max())
        assert ((diff - dx[:, k].double()).abs() <= tol).all()


def test_offsets_past_32_bits():
    """A matrix of more than 2^32 entries: its last rows are its own."""
    V, H, rows = 1_050_000, 4104, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    tail = (torch.randn(300, H, generator=g, device="cuda") * 0.1).bfloat16()
    w[-300:] = tail
    x = torch.randn(rows, H, generator=g, device="cuda").bfloat16()
    t = torch.tensor([V - 1, V - 299, 5], dtype=torch.int32, device="cuda")
    loss, lse = run_loss(x, w, t)
    z = x.double() @ tail.double().T
    want = torch.logsumexp(torch.cat([z, torch.full((rows, 1), float(V - 300), device="cuda").double().log()], 1), 1)
    dz = (H + 2) * 2.0 ** -23 * (x.double().abs() @ tail.double().abs().T).max(dim=1).values
    assert ((lse.double() - want).abs() <= dz + 2.0 ** -18).all()
    at = torch.stack([z[0, 299], z[1, 1], torch.zeros((), device="cuda").double()])
    assert ((loss.double() - (want - at)).abs() <= 2 * dz + 2.0 ** -18).all()
    grad = torch.ones(rows, device="cuda")
    dx, dw = run_grad(x, w, t, lse, grad)
    p = torch.exp(z - lse.double()[:, None])
    p[0, 299] -= 1
    p[1, 1] -= 1
    want_w = p.T @ x.double()
    tol = 2.0 ** -7 * (p.abs().T @ x.double().abs()) + 1e-6  # P's rounding, the result's and dz, 2^-9 each at most
    assert ((dw[-300:].double() - want_w).abs() <= tol).all()
    u = torch.exp(-lse.double())  # every other id's
    want_0 = (u[:, None] * x.double()).sum(0)
    assert ((dw[:5].double() - want_0).abs() <= 2.0 ** -7 * (u[:, None] * x.double().abs()).sum(0) + 1e-6).all()
    assert ((dx.double() - p @ tail.double()).abs() <= 2.0 ** -7 * (p.abs() @ tail.double().abs()) + 1e-6).all()


@pytest.mark.parametrize("same", [1, 8, 40])
@pytest.mark.parametrize("rows", [40, 300])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_target_entries_are_not_rounded(dtype, rows, same):
    """Gradients whose mantissa lies half way between two values of the type: rounded, a
    target's entry (nearly -1 here) would put 2^-8 (f16: 2^-11) of itself on all of its
    row's gradient. The results' own rounding has no such lean: over N entries it leaves
    about 0.6 / sqrt(N) of that, below 0.05."""
    V, H = 4000, 512
    half = torch.finfo(DT[dtype]).eps / 2
    x, w, t, _ = make(15, rows, V, H, dtype, spread=0.5, ignored=0.0)
    x = x * 0.1
    # up to eight rows a run of 32 ids (at most 299 * 13 + 5 = 3,892)
    t = torch.arange(rows, device="cuda").int() // same * (13 if same == 1 else 33) + 5
    grad = torch.full((rows,), 1 + half, device="cuda") * torch.where(torch.arange(rows, device="cuda") % 2 == 0, -4.0, 4.0)
    if same > 1:
        grad = grad.abs()
    _, lse = run_loss(x, w, t)
    dx, dw = check_grad(x, w, t, lse, grad)
    want_x, want_w = L.head_loss_grad(x, w, t, lse, grad)
    # (runs of 32 ids with more than eight rows keep the roundings of the rest)
    pairs = [(dx, want_x)] + ([(dw[t.long().unique()], want_w[t.long().unique()])] if same <= 8 else [])
    for got, want in pairs:
        lean = ((got.double() - want) * want).sum() / want.square().sum()
        assert abs(lean.item()) < 0.25 * half, lean.item() / half


@pytest.mark.parametrize("rows", [15, 16, 17, 32, 33, 48, 240, 241, 255, 272, 273, 512, 513, 1024, 1281])
def test_row_tiles(rows):
    """Tiles of 16 to 256 hidden rows, and one more than fill them."""
    x, w, t, grad = make(16, rows, 300, 72, "f16" if rows % 2 else "bf16")
    _, lse = check_loss(x, w, t)
    check_grad(x, w, t, lse, grad)


@pytest.mark.parametrize("H", [8, 120, 128, 136, 248, 256, 264, 392, 1024, 1032, 2048])
def test_widths(H):
    x, w, t, grad = make(17, 70, 600, H, "bf16")
    _, lse = check_loss(x, w, t)
    check_grad(x, w, t, lse, grad)


@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** -60, 2.0 ** 60, 2.0 ** 110])
def test_gradients_at_the_ends_of_fp32(scale):
    x, w, t, grad = make(18, 40, 300, 64, "bf16")
    _, lse = run_loss(x, w, t)
    check_grad(x, w, t, lse, grad * scale)


def test_nonfinite_gradients_reach_what_they_are_part_of():
    x, w, t, grad = make(19, 40, 300, 64, "bf16", ignored=0.0)
    _, lse = run_loss(x, w, t)
    grad[3], grad[30] = NAN, float("inf")
    dx, dw = run_grad(x, w, t, lse, grad)
    bad = ~torch.isfinite(dx).all(dim=1)
    assert bad.nonzero()[:, 0].tolist() == [3, 30] and not torch.isfinite(dw).any()
    t[3] = t[30] = -1  # ignored, they are nobody's
    dx, dw = run_grad(x, w, t, lse, grad)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


def test_many_pieces_and_a_narrow_last_one():
    """62 pieces of the vocabulary, the last of 576 ids, where dX's sums are split in two
    and the second part has nothing of it."""
    rows, V, H = 16_400, 1_000_000, 64
    g = torch.Generator(device="cuda").manual_seed(20)
    w = (torch.randn(V, H, generator=g, device="cuda") / 4).bfloat16()
    x = torch.randn(rows, H, generator=g, device="cuda").bfloat16()
    t = torch.randint(0, V, (rows,), generator=g, device="cuda").int()
    t[::5] = V - 1 - t[::5] % 500  # some in the last piece
    grad = torch.full((rows,), 0.5, device="cuda")
    loss, lse = run_loss(x, w, t)
    dx, dw = run_grad(x, w, t, lse, grad)
    x64, want_x, total = x.double(), torch.zeros(rows, H, device="cuda", dtype=torch.float64), None
    for lo in range(0, V, 50_000):
        part = w[lo:lo + 50_000].double()
        z = x64 @ part.T
        total = torch.logsumexp(z, 1) if total is None else torch.logaddexp(total, torch.logsumexp(z, 1))
        p = torch.exp(z - lse.double()[:, None])
        here = ((t >= lo) & (t < lo + 50_000)).nonzero()[:, 0]
        p[here, t[here].long() - lo] -= 1.0
        p *= 0.5
        want_x += p @ part
        want = p.T @ x64
        got = dw[lo:lo + 50_000].double()
        # two roundings of 2^-9 in the mean square at most, the sums' far below
        assert (got - want).norm() < 2.0 ** -8 * want.norm(), lo
        if lo + 50_000 >= V:
            assert (got[-576:] - want[-576:]).norm() < 2.0 ** -8 * want[-576:].norm()
    assert (lse.double() - total).abs().max() < 1e-4
    assert (dx.double() - want_x).norm() < 2.0 ** -8 * want_x.norm()


@pytest.mark.parametrize("rows", [7, 40, 300])
@pytest.mark.parametrize("apart", [20.0, 100.0, 1000.0])
def test_rows_far_apart(rows, apart):
    """Logits of neighbouring rows that lie far above and below each other: a row's sum
    does not vanish under another's reference."""
    x, w, t, grad = make(21, rows, 700, 64, "bf16")
    w[:, 0] = 1.0
    x[:, 0] = (torch.arange(rows, device="cuda") % 5 - 2).to(x.dtype) * apart
    _, lse = check_loss(x, w, t)
    check_grad(x, w, t, lse, grad)
