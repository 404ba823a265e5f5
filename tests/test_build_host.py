"""The build refuses a compiler whose register counts the wide 4-bit head cannot
be launched with (no GPU needed)."""
import os
import shutil

import pytest

from sampling_row_fp32_gb300 import build

needs_nvcc = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc is needed to build the library")

REPORT = """ptxas info    : 0 bytes gmem
ptxas info    : Compiling entry function '_ZN3sel11head_kernelI6__halfLi64EEEv' for 'sm_103a'
ptxas info    : Function properties for _ZN3sel11head_kernelI6__halfLi64EEEv
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used {} registers, used 16 barriers
ptxas info    : Compiling entry function '_ZN3sel12other_kernelEv' for 'sm_103a'
ptxas info    : Used 40 registers
"""


def test_registers_of_the_wide_head():
    build.check_registers("a.cu", REPORT.format(72), 72)
    with pytest.raises(RuntimeError, match="72 registers.*64"):
        build.check_registers("a.cu", REPORT.format(64), 72)
    with pytest.raises(RuntimeError, match="no head_kernel"):
        build.check_registers("a.cu", REPORT.replace("head_kernel", "tail_kernel"), 72)


@needs_nvcc
def test_the_build_checks_them(monkeypatch, tmp_path):
    """A count that the compiler does not give ends the build with the reason."""
    only = [s for s in build.sources() if s.endswith("sel_head_many_f16.cu")]
    monkeypatch.setattr(build, "sources", lambda: only)
    monkeypatch.setattr(build, "launch_registers", lambda: 71)
    with pytest.raises(RuntimeError, match="other than 71 registers"):
        build.build(out=str(tmp_path / "libsel.so"))
