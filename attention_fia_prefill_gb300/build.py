"""Builds libfia.so (the C-ABI library) in-tree with nvcc for sm_103a, and the
compiled Python binding of the paged-serving operators on top of it.

Each translation unit compiles in parallel; the .cu objects link into one
shared library next to this file (_lib/libfia.so), the binding into
_lib/_fia_paged.so, which needs libfia.so and the installed torch (where there
is none, libfia.so alone is built: its callers need the CUDA toolkit only).
Rebuilds only what is older than its sources and headers, and a binding built
against another torch.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libfia.so")
EXT = os.path.join(OUT_DIR, "_fia_paged.so")
EXT_TORCH = os.path.join(OUT_DIR, "_fia_paged.torch")   # the torch that the binding was built against
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


def _torch():
    """(folder, version) of the installed torch with CUDA, located without importing it, or None."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    where = spec.submodule_search_locations[0]
    if not os.path.exists(os.path.join(where, "lib", "libtorch_cuda.so")):
        return None
    with open(os.path.join(where, "version.py")) as f:
        return where, re.search(r"^__version__\s*=\s*['\"]([^'\"]+)", f.read(), re.M).group(1)


def _newer(target, files) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target) for f in files)


def _lib_current() -> bool:
    files, headers = _inputs()
    return _newer(LIB, files + headers + [os.path.abspath(__file__)])


def ext_torch_version() -> str:
    """Version of the torch that the binding was built against ("": no binding)."""
    if not os.path.exists(EXT) or not os.path.exists(EXT_TORCH):
        return ""
    with open(EXT_TORCH) as f:
        return f.read().strip()


def _ext_current(torch) -> bool:
    headers = [os.path.join(ROOT, "include", "fia.h")]
    return ext_torch_version() == torch[1] and _newer(EXT, headers + [EXT_SOURCE, os.path.abspath(__file__)])


def up_to_date() -> bool:
    torch = _torch()
    return _lib_current() and (torch is None or _ext_current(torch))


def _ext_commands(cc, torch):
    """(compile, link) commands of the binding: host code against the headers of torch (its folder), Python and the
    CUDA toolkit."""
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
    torch = _torch()
    want_lib = force or not _lib_current()
    want_ext = torch is not None and (force or not _ext_current(torch))
    if torch is None and verbose:
        print("no torch with CUDA here: libfia.so is built without the Python binding of the paged-serving operators")
    if not want_lib and not want_ext:
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

    with cf.ThreadPoolExecutor(max_workers=len(files) + 1) as ex:
        if want_ext:
            ext_compile, ext_link = _ext_commands(cc, torch[0])
            ext = ex.submit(_run, ext_compile, f"compiling {EXT_SOURCE}", verbose)
        if want_lib:
            tmp = LIB + ".tmp"
            _run([cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *ex.map(compile_one, files)], "link")
            os.replace(tmp, LIB)
        if want_ext:
            ext.result()
            _run(ext_link, "binding link")
            if os.path.exists(EXT_TORCH):
                os.remove(EXT_TORCH)
            os.replace(EXT + ".tmp", EXT)
            with open(EXT_TORCH, "w") as f:
                f.write(torch[1] + "\n")
    return LIB


if __name__ == "__main__":
    import sys
    print(build(verbose=True, force="--force" in sys.argv))
