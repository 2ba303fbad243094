"""Build step of the CUDA library: compiles csrc/*.cu for sm_103a with nvcc and
links them into ``libnmspmv.so`` next to this file (in-tree, never installed),
and, where PyTorch is installed, builds the compiled half of decode.py against it.

The translation units are compiled in parallel; nothing is rebuilt when the
library is newer than every source and header, and the binding newer than its own
and built for the running Python and PyTorch.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import platform
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libnmspmv.so")
# the compiled half of decode.py: tensors to arguments of the library's calls
EXT_PATH = os.path.join(HERE, "_decode_ext.so")
EXT_SOURCE = os.path.join(CSRC, "binding.cpp")

SOURCES = ["api.cu", "spmv.cu", "spmm.cu", "spmm_b2.cu", "spmm_b4.cu", "spmm_b6.cu", "spmm_b8.cu",
           "spmm24.cu", "gemv.cu", "pack.cu", "check_noalloc.cu", "prefill.cu", "rope_cache.cu",
           "attend.cu", "attend_wide_fp16.cu", "attend_wide_e4m3.cu", "attend_wide_int8.cu",
           "verify.cu", "decode_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-Wall", f"-I{INCLUDE}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def _library_inputs() -> list[str]:
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    files += glob.glob(os.path.join(INCLUDE, "*.h"))
    return files


def _inputs() -> list[str]:
    return _library_inputs() + [EXT_SOURCE]


def _newer(made: str, files: list[str]) -> bool:
    return os.path.exists(made) and all(os.path.getmtime(f) <= os.path.getmtime(made) for f in files)


def _python() -> str | None:
    """What the binding is built for, this Python and PyTorch; None without PyTorch,
    which the library itself does not need."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # not installed as a package
        version = spec.origin
    return f"{sys.implementation.cache_tag} {platform.machine()} torch {version}"


def _stamp() -> str:
    path = os.path.join(BUILD_DIR, "binding.for")
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read()


def library_up_to_date() -> bool:
    return _newer(LIB_PATH, _library_inputs())


def binding_up_to_date() -> bool:
    """Whether there is a binding for this Python and PyTorch (or nothing to build one for)."""
    want = _python()
    return want is None or (_newer(EXT_PATH, [EXT_SOURCE] + glob.glob(os.path.join(INCLUDE, "*.h")))
                            and _stamp() == want)


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _ext_command(out: str) -> tuple[list[str], list[str]]:
    """(compile, link) commands of the binding for the running Python and PyTorch."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(BUILD_DIR, "binding.o")
    cxx = os.environ.get("CXX") or "g++"
    compile_ = [cxx, "-std=c++17", "-O2", "-fPIC", "-Wall", f"-I{INCLUDE}",
                "-isystem", os.path.join(root, "include"),
                "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                "-isystem", os.path.join(cuda, "include"),
                "-isystem", sysconfig.get_paths()["include"],
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                "-c", EXT_SOURCE, "-o", obj]
    link = [cxx, "-shared", "-o", out, obj, f"-L{os.path.dirname(LIB_PATH)}",
            "-l:" + os.path.basename(LIB_PATH), "-Wl,-rpath,$ORIGIN",
            f"-L{os.path.join(root, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    return compile_, link


def _started(cmd: list[str]) -> subprocess.Popen:
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _linked(cmd: list[str], tmp: str, path: str) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link if needed, the binding too where PyTorch is there; returns the
    library path."""
    library = force or not library_up_to_date()
    binding = _python() is not None and (force or not binding_up_to_date())
    if not library and not binding:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    exe = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    ext_tmp = EXT_PATH + ".tmp"
    ext = None
    procs = []
    for src in SOURCES if library else []:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [exe, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        procs.append((src, obj, _started(cmd)))
    if binding:
        ext_compile, ext_link = _ext_command(ext_tmp)
        ext = _started(ext_compile)
    objs, errors = [], []
    for src, obj, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            errors.append(f"--- {src} ---\n{out}")
        elif verbose or ptxas_info:
            sys.stdout.write(out)
        objs.append(obj)
    if ext:
        out, _ = ext.communicate()
        if ext.returncode != 0:
            errors.append(f"--- {os.path.basename(EXT_SOURCE)} ---\n{out}")
    if errors:
        raise RuntimeError("compilation failed:\n" + "\n".join(errors))
    if library:
        tmp = LIB_PATH + ".tmp"
        _linked([exe, *ARCH, "-shared", "-o", tmp, *objs], tmp, LIB_PATH)
    if binding:
        _linked(ext_link, ext_tmp, EXT_PATH)
        with open(os.path.join(BUILD_DIR, "binding.for"), "w") as f:
            f.write(_python())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, ptxas_info="-v" in sys.argv))
