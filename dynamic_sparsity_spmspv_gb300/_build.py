"""Builds libdbspmspv.so in-tree (dynamic_sparsity_spmspv_gb300/_build/).

nvcc compiles the CUDA translation unit for sm_103a only; g++ compiles the
host builder; both run in parallel and nvcc links the shared library against
the static CUDA runtime.  Beside it, where torch is installed, g++ builds _dbsops.so,
the Python binding of the decoding step's operators; the library needs no torch
and is linked whatever comes of the binding.
"""
from __future__ import annotations

import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "_build")
LIB = os.path.join(OUT, "libdbspmspv.so")
OPS = os.path.join(OUT, "_dbsops.so")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")

CUDA_HOME = os.environ.get("CUDA_HOME", "/usr/local/cuda")
NVCC = os.path.join(CUDA_HOME, "bin", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]

SOURCES_CU = ["kernels.cu", "spmv.cu", "build_gpu.cu", "w4.cu", "rotary.cu", "norm.cu", "attention.cu", "window.cu", "pages.cu", "logits.cu"]
SOURCES_CPP = ["matrix.cpp"]


def _torch() -> tuple[str, str] | None:
    """Where torch is installed, and a line that names its version and Python's,
    without importing it; None where there is none."""
    import importlib.metadata
    import importlib.util
    import sysconfig
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    where = os.path.dirname(spec.origin)
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = ""
    return where, f"{where} {version} {sysconfig.get_config_var('SOABI')}"


def _fresh(path: str) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= _newest_input()


def _built_against() -> str:
    """The torch that the binding was built against."""
    try:
        with open(OPS + ".torch") as f:
            return f.read()
    except OSError:
        return ""


def _newest_input() -> float:
    """Latest modification time over every source and header the library is
    built from (all of csrc/ and include/), so that an edited header always
    triggers a rebuild."""
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp", ".h", ".cuh"))]
    paths += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return max(os.path.getmtime(p) for p in paths)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT, exist_ok=True)
    torch = _torch()
    lib = force or not _fresh(LIB)
    ops = torch is not None and (force or not _fresh(OPS) or _built_against() != torch[1])
    if not lib and not ops:
        return LIB
    import sysconfig
    procs = []
    objs = []

    def start(cmd):
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))

    for src in SOURCES_CU if lib else []:
        obj = os.path.join(OUT, src + ".o")
        cmd = [NVCC, *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
               "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        start(cmd)
        objs.append(obj)
    for src in SOURCES_CPP if lib else []:
        obj = os.path.join(OUT, src + ".o")
        start(["g++", "-O2", "-std=c++17", "-fPIC", "-pthread", "-Wall", "-I", INCLUDE,
               "-I", os.path.join(CUDA_HOME, "include"), "-c", os.path.join(CSRC, src), "-o", obj])
        objs.append(obj)
    ops_obj = os.path.join(OUT, "binding.cpp.o")
    if ops:
        start(["g++", "-O1", "-std=c++17", "-fPIC", "-Wall", "-I", os.path.join(torch[0], "include"),
               "-I", sysconfig.get_paths()["include"], "-I", os.path.join(CUDA_HOME, "include"),
               "-c", os.path.join(CSRC, "binding.cpp"), "-o", ops_obj])
    failed = []
    for cmd, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode != 0:
            print(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(cmd)
    if lib and not any(obj in cmd for cmd in failed for obj in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-lpthread"])
        os.replace(tmp, LIB)
    if failed:
        raise RuntimeError("dbspmspv build failed:\n" + "\n".join(" ".join(cmd) for cmd in failed))
    if ops:
        tmp = OPS + f".tmp{os.getpid()}"
        subprocess.check_call(["g++", "-shared", "-o", tmp, ops_obj, "-L", OUT, "-l:libdbspmspv.so", "-Wl,-rpath,$ORIGIN",
                               "-L", os.path.join(torch[0], "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
        os.replace(tmp, OPS)
        with open(OPS + ".torch", "w") as f:
            f.write(torch[1])
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
