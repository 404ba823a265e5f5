"""The binding of the operators around selection refuses sizes that the library's
32-bit arguments do not hold (no GPU needed: the tensors have no memory)."""
import pytest
import torch

from sampling_row_fp32_gb300 import binding as B

BIG = 2 ** 32 + 3


def t(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


class Reached:
    def __getattr__(self, name):
        def call(*args):
            raise AssertionError(f"{name} was called")
        return call


@pytest.fixture(autouse=True)
def no_gpu(monkeypatch):
    monkeypatch.setattr(B, "_device", lambda *tensors: 0)
    monkeypatch.setattr(B, "_on_stream", lambda stream, dev: 0)
    monkeypatch.setattr(B, "_lib", Reached())


def sample(rows, V):
    f = t(rows, dtype=torch.float32)
    B.sel_sample16(t(rows, V), None, None, None, None, f, t(rows, dtype=torch.int32), f)


@pytest.mark.parametrize("call", [
    lambda: sample(BIG, 1),
    lambda: sample(2, BIG),
    lambda: B.sel_head_w4(t(BIG, 64), t(5, 32, dtype=torch.uint8), t(5, 1), None, 64, t(BIG, 5)),
    lambda: B.sel_head_w4(t(2, 64), t(BIG, 32, dtype=torch.uint8), t(BIG, 1), None, 64, t(2, BIG)),
    lambda: B.sel_head_w4(t(2, 2 ** 32), t(5, 2 ** 31, dtype=torch.uint8), t(5, 2 ** 26), None, 64, t(2, 5)),
    lambda: B.sel_embed(t(BIG, dtype=torch.int32), t(5, 1), 1.0, t(BIG, 1)),
    lambda: B.sel_embed(t(3, dtype=torch.int32), t(BIG, 1), 1.0, t(3, 1)),
    lambda: B.sel_embed(t(3, dtype=torch.int32), t(1, BIG), 1.0, t(3, BIG)),
    lambda: B.sel_embed_w4(t(BIG, dtype=torch.int32), t(5, 16, dtype=torch.uint8), t(5, 1), None, 32, 1.0, t(BIG, 32)),
    lambda: B.sel_embed_w4(t(3, dtype=torch.int32), t(BIG, 16, dtype=torch.uint8), t(BIG, 1), None, 32, 1.0, t(3, 32)),
])
def test_sizes_past_32_bits_are_refused(call):
    with pytest.raises(ValueError):
        call()


def test_sizes_within_them_reach_the_library():
    with pytest.raises(AssertionError, match="sel_sample16 was called"):
        sample(2 ** 32 - 1, 1)
    with pytest.raises(AssertionError, match="sel_embed was called"):
        B.sel_embed(t(3, dtype=torch.int32), t(5, 1), 1.0, t(3, 1))
