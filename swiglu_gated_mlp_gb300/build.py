"""In-tree build of libswiglu.so (nvcc, sm_103a only, no cmake).

Each CUDA translation unit is compiled in parallel into ``_build/`` beside this
file, then linked into ``libswiglu.so`` in this package directory with the
CUDA runtime linked statically and only the ``swiglu_*`` symbols exported. A
stamp of the sources and flags skips the work when nothing changed. Beside it
``torch_calls.cpp`` (Python calls for the installed PyTorch) becomes
``_torch_calls.so``, which uses libswiglu.so from the same directory. The C
library does not need it: without PyTorch, g++ or Python's headers it is left out.

    python -m swiglu_gated_mlp_gb300.build        # build (or check) the library
"""
from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libswiglu.so")
CALLS_PATH = os.path.join(PKG_DIR, "_torch_calls.so")
STAMP = os.path.join(BUILD_DIR, "libswiglu.stamp")

SOURCES = ["swiglu_api.cu", "pack.cu", "fused_large_m.cu", "fused_large_m_pair.cu", "fused_small_m.cu",
           "fused_sequential.cu", "fused_split_k.cu", "fused_resident_pair.cu", "backward_pair.cu",
           "backward_api.cu", "lora_shrink.cu", "lora_api.cu", "quantize.cu", "checkpoint.cu",
           "checkpoint_api.cu", "int8_gemm.cu", "int8_api.cu"]
CALLS_SOURCE = "torch_calls.cpp"
HEADERS = ["kernels.h", "ptx.cuh", "lora_lb.cuh", "int8.cuh", "api_shared.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                 "-Xptxas", "-v", "-I" + INCLUDE, "-I" + CSRC]
VERSION_SCRIPT = "{ global: swiglu_*; local: *; };\n"


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libswiglu")


def calls_built_for(torch) -> str:
    """What _torch_calls.so is built for: it uses the binary interfaces of PyTorch and of Python."""
    return f"PyTorch {torch.__version__}, Python {sysconfig.get_config_var('SOABI')}"


def _calls_flags() -> tuple | None:
    """Compiler and linker flags of _torch_calls.so, or None where it cannot be built."""
    try:
        import torch
    except ImportError:
        return None
    if not shutil.which("g++") or not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return None
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [os.path.join(base, "include"), os.path.join(base, "include/torch/csrc/api/include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    return (["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
             f'-DSWIGLU_BUILT_FOR="{calls_built_for(torch)}"',
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + ["-I" + i for i in include],
            ["-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
             "-Wl,-rpath," + os.path.join(base, "lib"), "-L" + BUILD_DIR, "-l:libswiglu.so", "-Wl,-rpath,$ORIGIN"])


def _stamp(nvcc: str) -> str:
    h = hashlib.sha256()
    h.update(repr(_calls_flags()).encode())
    for name in SOURCES + HEADERS + [CALLS_SOURCE]:
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(name.encode() + b"\0" + f.read())
    with open(os.path.join(INCLUDE, "swiglu.h"), "rb") as f:
        h.update(f.read())
    h.update(" ".join(CFLAGS).encode())
    h.update(subprocess.run([nvcc, "--version"], capture_output=True, text=True).stdout.encode())
    h.update(os.uname().machine.encode())
    return h.hexdigest()


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libswiglu.so if it is missing or stale; return its path."""
    nvcc = _nvcc()
    stamp = _stamp(nvcc)
    if not force and os.path.exists(LIB_PATH) and os.path.exists(STAMP):
        with open(STAMP) as f:
            was = f.read().split()
        # (a second word: _torch_calls.so was left out)
        if was and was[0] == stamp and (len(was) > 1 or os.path.exists(CALLS_PATH)):
            return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(name: str):
        obj = os.path.join(BUILD_DIR, name.replace(".cu", ".o"))
        cmd = [nvcc, "-c", os.path.join(CSRC, name), "-o", obj] + CFLAGS
        r = subprocess.run(cmd, capture_output=True, text=True)
        return name, obj, r

    calls_flags = _calls_flags()
    calls_obj = os.path.join(BUILD_DIR, CALLS_SOURCE.replace(".cpp", ".o"))

    def compile_calls():
        cmd = ["g++", "-c", os.path.join(CSRC, CALLS_SOURCE), "-o", calls_obj] + calls_flags[0]
        return subprocess.run(cmd, capture_output=True, text=True)

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(compile_calls) if calls_flags else None
        results = list(ex.map(compile_one, SOURCES))
        calls = calls.result() if calls else None
    log = []
    for name, _, r in results:
        log.append(f"==== {name}\n{r.stdout}{r.stderr}")
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {name}:\n{r.stdout}{r.stderr}")
    with open(os.path.join(BUILD_DIR, "ptxas.log"), "w") as f:
        f.write("\n".join(log))
    vs = os.path.join(BUILD_DIR, "exports.map")
    with open(vs, "w") as f:
        f.write(VERSION_SCRIPT)
    new_lib = os.path.join(BUILD_DIR, os.path.basename(LIB_PATH))
    cmd = [nvcc, "-shared", "-o", new_lib] + [o for _, o, _ in results] + ARCH + [
        "--cudart", "static", "-Xlinker", "--version-script=" + vs, "-Xlinker", "-z,defs",
        "-lpthread", "-ldl", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    new_calls = os.path.join(BUILD_DIR, os.path.basename(CALLS_PATH))
    if calls and calls.returncode == 0:
        calls = subprocess.run(["g++", "-shared", "-o", new_calls, calls_obj] + calls_flags[1], capture_output=True,
                               text=True)
    left_out = not calls or calls.returncode != 0
    if left_out:
        warnings.warn("_torch_calls.so is left out, so the 8-bit calls are made from Python: "
                      + (calls.stderr if calls else "it needs PyTorch, g++ and Python's headers"), RuntimeWarning)
    # in place together, after both links
    os.replace(new_lib, LIB_PATH)
    if not left_out:
        os.replace(new_calls, CALLS_PATH)
    elif os.path.exists(CALLS_PATH):
        os.remove(CALLS_PATH)
    with open(STAMP, "w") as f:
        f.write(stamp + (" without-calls" if left_out else "") + "\n")
    if verbose:
        print("\n".join(log))
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
