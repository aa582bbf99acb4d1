"""Build libarf.so (the CUDA library behind include/arf.h) for sm_103a, and
the module _torch_ops that calls it on torch tensors.

Each translation unit under csrc/ is compiled by nvcc (torch_ops.cpp by the
host compiler against torch's headers) in parallel, then the objects are
linked into a shared library next to this file with the CUDA runtime linked
statically, and the module beside it. The library needs no torch: where there
is none, it is built alone. Built in place; the outputs are git-ignored.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libarf.so")
TORCH_SOURCE = "torch_ops.cpp"
TORCH_LIB = os.path.join(PKG, "_torch_ops.so")
TORCH_STAMP = os.path.join(BUILD_DIR, "torch_ops.stamp")  # what the module was built against

SOURCES = ["arf_api.cu", "arf_launch_bf16.cu", "arf_launch_fp16.cu", "arf_static.cu", "arf_measure.cu",
           "arf_rotary.cu", "arf_decode.cu", "arf_decode_bf16.cu", "arf_decode_fp16.cu", "arf_pages.cu"]
GENCODE = "-gencode=arch=compute_103a,code=sm_103a"
# No fast-math and no automatic FMA contraction: the rank-order sum and the
# normalisation are written with explicit IEEE operations.
NVCC_FLAGS = [GENCODE, "-O3", "-std=c++17", "-lineinfo", "--fmad=false",
              "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libarf.so")


def _torch_stamp():
    """The interpreter and the torch that the module is bound to (by torch's
    C++ layout), or None without torch. Does not import torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    root = os.path.dirname(spec.origin)
    with open(os.path.join(root, "version.py")) as f:
        return "\n".join((sys.version, root, f.read()))


def _torch_commands(obj: str, out: str):
    """The commands that compile and link the module against torch."""
    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(root, "lib")
    compile_cmd = [cxx, "-O2", "-std=c++20", "-fPIC", "-fvisibility=hidden",
                   f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
                   *[x for d in inc for x in ("-isystem", d)], "-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj]
    link_cmd = [cxx, "-shared", "-o", out, obj, "-L", PKG, "-larf", "-L", lib, "-ltorch_python", "-ltorch_cuda",
                "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    return compile_cmd, link_cmd


def _newer(files, out) -> bool:
    return not os.path.exists(out) or any(os.path.getmtime(f) > os.path.getmtime(out) for f in files)


def _lib_stale() -> bool:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != TORCH_SOURCE]
    return _newer([f for f in files if os.path.isfile(f)] + [os.path.join(INCLUDE, "arf.h"), __file__], LIB)


def _module_stale(stamp) -> bool:
    if stamp is None:
        return False
    if _newer([os.path.join(CSRC, TORCH_SOURCE), os.path.join(INCLUDE, "arf.h"), __file__], TORCH_LIB):
        return True
    if not os.path.exists(TORCH_STAMP):
        return True
    with open(TORCH_STAMP) as f:
        return f.read() != stamp


def stale() -> bool:
    return _lib_stale() or _module_stale(_torch_stamp())


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link libarf.so and, where torch is installed, _torch_ops.so
    if they are missing or out of date."""
    stamp = _torch_stamp()
    lib, module = force or _lib_stale(), stamp is not None and (force or _module_stale(stamp))
    if not (lib or module):
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        said = _run(cmd, f"nvcc failed on {src}")
        if ptxas_info or verbose:
            sys.stderr.write(said)
        return obj

    torch_tmp = TORCH_LIB + ".tmp"
    if module:
        torch_compile, torch_link = _torch_commands(os.path.join(BUILD_DIR, "torch_ops.o"), torch_tmp)

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        torch_done = ex.submit(_run, torch_compile, f"compiler failed on {TORCH_SOURCE}") if module else None
        objs = list(ex.map(compile_one, SOURCES)) if lib else []
        if lib:
            tmp = LIB + ".tmp"
            _run([cc, GENCODE, "-shared", "-cudart", "static", "-o", tmp, *objs], "link failed")
            os.replace(tmp, LIB)
        if module:
            torch_done.result()
    if module:
        _run(torch_link, "link of _torch_ops failed")
        os.replace(torch_tmp, TORCH_LIB)
        with open(TORCH_STAMP, "w") as f:
            f.write(stamp)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
