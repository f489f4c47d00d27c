"""Build ``libspecverify.so`` in-tree with nvcc for sm_103a, and the bindings of its cache calls
(``_kvbind.so``) and of its log probabilities (``_lpbind.so``) with g++, all translation units in
parallel."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
#: Each translation unit with the files it is made of.
UNITS = {
    "specverify": [os.path.join(CSRC, "specverify.cu"), os.path.join(CSRC, "ff.cuh"),
                   os.path.join(INCLUDE, "specverify.h"),
                   os.path.join(INCLUDE, "specverify_debug.h")],
    "kvcache": [os.path.join(CSRC, "kvcache.cu"), os.path.join(CSRC, "kvattention.cuh"),
                os.path.join(INCLUDE, "specverify.h"), os.path.join(INCLUDE, "specverify_kv.h")],
    "kvwindow": [os.path.join(CSRC, "kvwindow.cu"), os.path.join(CSRC, "kvattention.cuh"),
                 os.path.join(INCLUDE, "specverify.h"), os.path.join(INCLUDE, "specverify_kv.h")],
    "logprobs": [os.path.join(CSRC, "logprobs.cu"), os.path.join(INCLUDE, "specverify.h"),
                 os.path.join(INCLUDE, "specverify_logprobs.h")],
}
LIB = os.path.join(HERE, "libspecverify.so")
#: The bindings, extension modules of this interpreter and its torch, with the files of each.
BINDINGS = {
    os.path.join(HERE, f"_{name}.so"): [os.path.join(CSRC, name + ".cpp"),
                                        os.path.join(CSRC, "bind.h"),
                                        os.path.join(INCLUDE, "specverify.h"),
                                        os.path.join(INCLUDE, header)]
    for name, header in (("kvbind", "specverify_kv.h"), ("lpbind", "specverify_logprobs.h"))}
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(home, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def bind_command(source: str, out: str) -> list[str]:
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    include = [sysconfig.get_paths()["include"], INCLUDE, os.path.join(torch, "include"),
               os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include")]
    return (["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-w"] + [f"-I{p}" for p in include]
            + ["-o", out, source, "-L" + os.path.join(torch, "lib"), "-ltorch_python",
               "-ltorch_cpu", "-lc10", "-lc10_cuda"])


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the CUDA library and the bindings unless they are newer than every
    source; of the library's units only those older than their files."""
    newer = lambda out, files: not force and os.path.exists(out) and (
        os.path.getmtime(out) >= max(os.path.getmtime(f) for f in files))
    lib_done = newer(LIB, [f for files in UNITS.values() for f in files])
    if lib_done and all(newer(*b) for b in BINDINGS.items()):
        return LIB
    folder = os.path.join(HERE, "_build")
    os.makedirs(folder, exist_ok=True)
    running = []
    for bind, files in BINDINGS.items():
        if newer(bind, files):
            continue
        tmp = bind + f".tmp{os.getpid()}"
        cmd = bind_command(files[0], tmp)
        running.append((cmd, subprocess.Popen(cmd), tmp, bind))
    for name, files in UNITS.items():
        obj = os.path.join(folder, name + ".o")
        if lib_done or newer(obj, files):
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
    if lib_done:
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc(), ARCH, "-shared", "-o", tmp]
                   + [os.path.join(folder, name + ".o") for name in UNITS], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    build(force=True, verbose="-v" in sys.argv)
    print(LIB)
