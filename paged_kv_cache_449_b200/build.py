"""Builds libpa.so in-tree with nvcc for sm_100a (B200).

The library is two translation units (csrc/pa_api.cu and csrc/pa_ops.cu plus
their headers), compiled side by side and linked against the static CUDA runtime
so it loads without a GPU or driver present.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
UNITS = [os.path.join(HERE, "csrc", name) for name in ("pa_api.cu", "pa_ops.cu")]
LIB = os.path.join(HERE, "libpa.so")
# The same sources with the test hooks of include/pa_test.h compiled in (for
# the tests of the kernels' bounded waits); never loaded by the product.
TEST_LIB = os.path.join(HERE, "libpa_test.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    found = shutil.which("nvcc")
    if found:
        return found
    return "/usr/local/cuda/bin/nvcc"


def sources() -> list[str]:
    return UNITS + sorted(glob.glob(os.path.join(HERE, "csrc", "*.cuh"))) + \
        sorted(glob.glob(os.path.join(ROOT, "include", "**", "*.h"), recursive=True))


def build(out: str = LIB, defines: dict | None = None, force: bool = False, verbose: bool = False) -> str:
    """Compile the library; skipped when `out` is newer than every source
    (each output file is built with one fixed set of defines)."""
    if not force and os.path.exists(out):
        if os.path.getmtime(out) >= max(os.path.getmtime(s) for s in sources()):
            return out
    flags = [*ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]
    flags += [f"-D{k}={v}" for k, v in (defines or {}).items()]
    if verbose:
        flags += ["-Xptxas", "-v"]
    tmp = f"{out}.tmp{os.getpid()}"
    objects = [f"{tmp}.{i}.o" for i in range(len(UNITS))]
    try:
        running = [subprocess.Popen([nvcc_path(), *flags, "-c", "-o", obj, src]) for src, obj in zip(UNITS, objects)]
        codes = [p.wait() for p in running]   # (every one is waited for, whatever the others did)
        for p, code in zip(running, codes):
            if code != 0:
                raise subprocess.CalledProcessError(code, p.args)
        subprocess.run([nvcc_path(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objects], check=True)
    finally:
        for obj in objects:
            if os.path.exists(obj):
                os.remove(obj)
    os.replace(tmp, out)
    return out


def build_test(force: bool = False) -> str:
    """libpa_test.so: the library with PA_TEST_HOOKS defined."""
    return build(TEST_LIB, defines={"PA_TEST_HOOKS": 1}, force=force)


if __name__ == "__main__":
    print(build(force=True))
