"""Build ``libspecverify.so`` in-tree with nvcc for sm_103a (its translation units in parallel)."""
from __future__ import annotations

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
#: Each translation unit with the files it is made of.
UNITS = {
    "specverify": [os.path.join(CSRC, "specverify.cu"), os.path.join(CSRC, "ff.cuh"),
                   os.path.join(INCLUDE, "specverify.h"),
                   os.path.join(INCLUDE, "specverify_debug.h")],
    "kvcache": [os.path.join(CSRC, "kvcache.cu"), os.path.join(INCLUDE, "specverify.h"),
                os.path.join(INCLUDE, "specverify_kv.h")],
}
LIB = os.path.join(HERE, "libspecverify.so")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(home, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the CUDA library unless it is newer than every source; of its
    units only those that are older than their files."""
    newer = lambda out, files: os.path.exists(out) and (
        os.path.getmtime(out) >= max(os.path.getmtime(f) for f in files))
    if not force and newer(LIB, [f for files in UNITS.values() for f in files]):
        return LIB
    folder = os.path.join(HERE, "_build")
    os.makedirs(folder, exist_ok=True)
    running = []
    for name, files in UNITS.items():
        obj = os.path.join(folder, name + ".o")
        if not force and newer(obj, files):
            continue
        tmp = obj + f".tmp{os.getpid()}"
        cmd = [nvcc(), ARCH, "-O3", "-lineinfo", "-std=c++17", "-c", "-Xcompiler", "-fPIC",
               "-I", INCLUDE, "-o", tmp, files[0]]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        running.append((cmd, subprocess.Popen(cmd), tmp, obj))
    failed = None
    for cmd, proc, tmp, obj in running:
        if proc.wait() == 0:
            os.replace(tmp, obj)
        else:
            failed = subprocess.CalledProcessError(proc.returncode, cmd)
    if failed:
        raise failed
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc(), ARCH, "-shared", "-o", tmp]
                   + [os.path.join(folder, name + ".o") for name in UNITS], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    build(force=True, verbose="-v" in sys.argv)
    print(LIB)
