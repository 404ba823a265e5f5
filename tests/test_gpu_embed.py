"""sel_embed and sel_embed_w4 on the GPU against 64-bit lookups."""
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


def some_ids(rng, n, V):
    ids = rng.integers(0, V, size=n, dtype=np.uint32)
    ids[rng.random(n) < 0.2] = B.SEL_INVALID_ID
    if n > 3:
        ids[:4] = [V - 1, 0, V, V - 1]  # the last row, the first, one past the end, a repeat
    return ids


def close(out, want, dtype):
    """One rounding of a value formed in fp32: half a step of the type plus
    half a step of fp32, each relative to the value (subnormal results: to the
    type's smallest step)."""
    rel = torch.finfo(dtype).eps / 2 + 2.0 ** -24
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    got = out.double().cpu().numpy()
    assert got.shape == want.shape
    assert (np.abs(got - want) <= rel * (1 + rel) * np.abs(want) + tiny).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,V,H,off", [(1, 5, 1, 0), (7, 33, 2049, 0), (49, 1000, 4096, 0), (3, 70, 256, 1),
                                       (1000, 257, 24, 0), (2, 3, 8, 0)])
def test_table(dtype, n, V, H, off):
    """off = 1 moves the table one element from its 16-byte boundary."""
    rng = np.random.default_rng(n + H)
    dt = DT[dtype]
    flat = torch.empty(V * H + off, dtype=dt, device="cuda")
    table = flat[off:].view(V, H)
    table.copy_(torch.from_numpy(rng.normal(0, 0.3, size=(V, H))))
    ids = some_ids(rng, n, V)
    scale = float(np.float32(np.sqrt(H)))
    out = torch.full((n, H), 7.0, dtype=dt, device="cuda")
    B.sel_embed(torch.from_numpy(ids.view(np.int32)).cuda(), table, scale, out)
    close(out, D.embed(ids, table.double().cpu().numpy(), scale), dt)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,V,H,group,zeros", [(1, 1, 32, 32, False), (49, 515, 4096, 64, False), (5, 77, 2880, 32, True),
                                               (600, 40, 128, 128, True)])
def test_w4(dtype, n, V, H, group, zeros):
    rng = np.random.default_rng(H + n)
    dt = DT[dtype]
    q = rng.integers(0, 256, size=(V, H // 2), dtype=np.uint8)
    s = torch.from_numpy(rng.uniform(-0.1, 0.1, size=(V, H // group))).to(dt)
    z = rng.integers(0, 256, size=(V, H // group), dtype=np.uint8) if zeros else None
    ids = some_ids(rng, n, V)
    out = torch.full((n, H), 7.0, dtype=dt, device="cuda")
    B.sel_embed_w4(torch.from_numpy(ids.view(np.int32)).cuda(), torch.from_numpy(q).cuda(), s.cuda(),
                   None if z is None else torch.from_numpy(z).cuda(), group, 3.5, out)
    close(out, D.embed(ids, D.dequantise(q, s.double().numpy(), z, group), 3.5), dt)


def test_ids_of_any_shape_and_offsets_past_32_bits():
    """Emitted [S][K + 1] ids, and a table of more than 2^32 elements."""
    V, H = 1_100_000, 4096
    table = torch.empty(V, H, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([[V - 1, -1, 0], [V - 2, V - 1, 5]], dtype=torch.int32, device="cuda")
    for i in (0, 5, V - 2, V - 1):
        table[i] = torch.arange(H, device="cuda") * 0.5 + (i % 7)
    out = torch.full((2, 3, H), 7.0, dtype=torch.bfloat16, device="cuda")
    B.sel_embed(ids, table, 1.0, out)
    assert torch.equal(out[0, 0], table[V - 1]) and torch.equal(out[1, 0], table[V - 2])
    assert torch.equal(out[0, 2], table[0]) and torch.equal(out[1, 2], table[5])
    assert not out[0, 1].any()


def test_no_ids():
    out = torch.full((0, 16), 7.0, device="cuda")
    B.sel_embed(torch.empty(0, dtype=torch.int32, device="cuda"), torch.zeros(3, 16, device="cuda"), 1.0, out)
