"""Builds libfia.so (the C-ABI library) in-tree with nvcc for sm_103a, and the
compiled Python binding of the paged-serving operators on top of it.

Each translation unit compiles in parallel; the .cu objects link into one
shared library next to this file (_lib/libfia.so), the binding into
_lib/_fia_paged.so, which needs libfia.so and the installed torch.  Rebuilds
only when a source or header is newer than the libraries.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libfia.so")
EXT = os.path.join(OUT_DIR, "_fia_paged.so")
EXT_SOURCE = os.path.join(CSRC, "py_paged.cpp")
SOURCES = ["fia_api.cu", "prefill.cu", "prefill_pair.cu", "bsa_fp8.cu", "decode.cu", "decode_d64.cu", "decode_gqa.cu", "decode_noalloc.cu",
           "mla.cu", "paged_api.cu", "paged.cu", "span_decode.cu", "span_wide.cu", "prefill_window.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xcompiler", "-fvisibility=hidden", "-cudart", "shared"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(ROOT, "include", "fia.h"))
    return files, headers


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(EXT):
        return False
    files, headers = _inputs()
    t = min(os.path.getmtime(LIB), os.path.getmtime(EXT))
    return all(os.path.getmtime(f) <= t for f in files + headers + [EXT_SOURCE, os.path.abspath(__file__)])


def _ext_commands(cc):
    """(compile, link) commands of the binding: host code against the headers of torch (located without importing
    it), Python and the CUDA toolkit."""
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(cc)))
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    lib = os.path.join(torch, "lib")
    obj = os.path.join(OUT_DIR, "py_paged.o")
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    return ([cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *(f"-I{i}" for i in inc), "-c", EXT_SOURCE, "-o", obj],
            [cxx, "-shared", "-o", EXT + ".tmp", obj, "-L" + OUT_DIR, "-lfia", "-L" + lib, "-ltorch_python", "-ltorch_cpu",
             "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib])


def _run(cmd, what, verbose=False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout, r.stderr)


def build(verbose: bool = False, force: bool = False, extra_flags=None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    files, _ = _inputs()
    cc = nvcc()
    extra = list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src).replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
        _run(cmd, f"nvcc for {src}", verbose)
        return obj

    ext_compile, ext_link = _ext_commands(cc)
    with cf.ThreadPoolExecutor(max_workers=len(files) + 1) as ex:
        ext = ex.submit(_run, ext_compile, f"compiling {EXT_SOURCE}", verbose)
        objs = list(ex.map(compile_one, files))
        ext.result()
    tmp = LIB + ".tmp"
    _run([cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs], "link")
    os.replace(tmp, LIB)
    _run(ext_link, "binding link")
    os.replace(EXT + ".tmp", EXT)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(verbose=True, force="--force" in sys.argv))
