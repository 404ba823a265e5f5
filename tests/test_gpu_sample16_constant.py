"""sel_sample16 on the GPU: constant rows of the widest kind, one CTA a row.

Every lane of the pass that looks for the drawn id then counts all the ids that
it sees, up to 260 in a half: 64 whole vectors and an end vector of the row."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from sampling_row_fp32_gb300 import binding as B

pytestmark = pytest.mark.gpu

ROWS = 130  # one CTA a row: fewer rows than SMs, more than half of them


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def uniforms(V, skew):
    """Uniforms over the whole range, and those next to the borders between the
    runs of a CTA's 32 warps and to the row's ends."""
    run = -(-(-(-(V + skew) // 8)) // 32)
    at = [min(V, max(0, 8 * w * run - skew) + d) for w in range(1, 33) for d in (-2, -1, 0, 1, 2)] + [0, 1, V - 2, V - 1, V]
    u = [np.float32(a / V) for a in at]
    u += [np.nextafter(x, np.float32(0)) for x in u] + [np.nextafter(x, np.float32(1)) for x in u]
    u += list(np.linspace(0, 1, 400, endpoint=False, dtype=np.float32)) + [np.float32(1 - 2.0 ** -24)]
    return np.unique(np.array(u, dtype=np.float32).clip(0, np.float32(1 - 2.0 ** -24)))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("V,off,pad", [(517_001, 3, 0), (520_001, 5, 0), (524_201, 0, 0), (524_201, 0, 7), (524_208, 0, 1),
                                       (524_208, 1, 8), (524_208, 7, 8), (516_400, 3, 8), (400_003, 1, 0)])
def test_constant_rows(dtype, V, off, pad):
    ld = V + pad
    flat = torch.full((off + ROWS * ld,), float("nan"), dtype=dtype, device="cuda")
    x = flat[off:].view(ROWS, ld)[:, :V]
    x.fill_(-1.5)
    u = np.concatenate([uniforms(V, s) for s in sorted({(off + r * ld) % 8 for r in range(8)})])
    u = np.unique(u)
    u = np.resize(u, -(-u.size // ROWS) * ROWS)  # (the first ones again)
    # every weight is 1: the first id whose count exceeds u V, in whole numbers
    want = np.array([int(Fraction(float(v)) * V) for v in u], dtype=np.int64)
    # each uniform in rows of all eight alignments
    for turn in range(8):
        v = np.roll(u, turn)
        got, probs = [], []
        for lo in range(0, v.size, ROWS):
            ids = torch.full((ROWS,), -7, dtype=torch.int32, device="cuda")
            pr = torch.full((ROWS,), -7.0, device="cuda")
            B.sel_sample16(x, None, None, None, None, torch.from_numpy(v[lo:lo + ROWS]).cuda(), ids, pr)
            got.append(ids)
            probs.append(pr)
        ids = torch.cat(got).cpu().numpy().astype(np.int64)
        w = np.roll(want, turn)
        assert np.array_equal(ids, w), (int((ids != w).sum()), ids[ids != w][:8], w[ids != w][:8])
        assert (torch.cat(probs).cpu().numpy() == np.float32(1.0 / V)).all()
