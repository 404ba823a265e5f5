"""Build the C-ABI library ``libsel.so`` in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` is compiled to an object in parallel, then linked into
``_build/libsel.so`` (CUDA runtime linked statically, so the library depends
only on the driver). Run ``python -m sampling_row_fp32_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import re
import shutil
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libsel.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsel.so")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def launch_registers() -> int:
    """The registers a thread that the wide head's split between its warps
    counts on (csrc/sel_head_many.cuh)."""
    text = open(os.path.join(CSRC, "sel_head_many.cuh")).read()
    return int(re.search(r"kLaunchRegs = (\d+)", text).group(1))


def check_registers(src: str, report: str, want: int) -> None:
    """Raise unless every head_kernel in the assembler's report (-Xptxas -v)
    takes `want` registers a thread: with another number, which another compiler
    may choose, the library refuses every call of it."""
    found = {}
    name = None
    for line in report.splitlines():
        if m := re.search(r"Compiling entry function '([^']+)'", line):
            name = m.group(1)
        elif name and (m := re.search(r"Used (\d+) registers", line)):
            found[name] = int(m.group(1))
            name = None
    heads = {n: r for n, r in found.items() if "head_kernel" in n}
    if not heads:
        raise RuntimeError(f"{os.path.basename(src)}: the assembler reported no head_kernel")
    wrong = {n: r for n, r in heads.items() if r != want}
    if wrong:
        raise RuntimeError(f"{os.path.basename(src)}: kernels of other than {want} registers a thread, on which the "
                           f"split between their warps (kLaunchRegs) counts: {wrong}")


def _inputs() -> list[str]:
    files = sources()
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags: tuple[str, ...] = (),
          out: str | None = None) -> str:
    """Compile and link libsel.so unless it is newer than every source.
    `out` (with `extra_flags`, e.g. -D tuning overrides) builds a separate
    copy at that path instead, in its own object directory."""
    lib = out or LIB
    if not force and out is None and up_to_date():
        return LIB
    objdir = BUILD if out is None else os.path.splitext(out)[0] + "_obj"
    os.makedirs(objdir, exist_ok=True)
    cc = nvcc()
    objs = []

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
        counted = os.path.basename(src).startswith("sel_head_many")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *(["-Xptxas", "-v"] if counted else []), *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if counted:
            check_registers(src, r.stdout + r.stderr, launch_registers())
        if verbose:
            sys.stdout.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, sources()))
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=objdir)
    os.close(fd)
    try:
        cmd = [cc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    finally:
        if os.path.exists(tmp):
            os.unlink(tmp)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
