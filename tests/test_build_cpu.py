"""What build() compiles and when, with the compilers' commands recorded instead
of run: the C library needs the CUDA toolkit alone, the Python binding the torch
that is installed."""
import importlib.util
import os
import types

import pytest

from attention_fia_prefill_gb300 import build as b


@pytest.fixture
def bench(tmp_path, monkeypatch):
    """An empty output folder, a recorded _run, and a torch whose version (None: no torch) the test sets."""
    ran, torch = [], types.SimpleNamespace(version="2.9.1+cu130", cuda=True)
    out = tmp_path / "_lib"

    def run(cmd, what, verbose=False):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    def find_spec(name, *a):
        if name != "torch":
            return real(name, *a)
        if torch.version is None:
            return None
        folder = tmp_path / "torch"
        (folder / "lib").mkdir(parents=True, exist_ok=True)
        if torch.cuda:
            (folder / "lib" / "libtorch_cuda.so").write_text("")
        (folder / "version.py").write_text(f"__all__ = ['__version__']\n__version__ = '{torch.version}'\ncuda = '13.0'\n")
        return types.SimpleNamespace(submodule_search_locations=[str(folder)])

    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", find_spec)
    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(b, "OUT_DIR", str(out))
    for name, file in (("LIB", "libfia.so"), ("EXT", "_fia_paged.so"), ("EXT_TORCH", "_fia_paged.torch")):
        monkeypatch.setattr(b, name, str(out / file), raising=False)
    return types.SimpleNamespace(ran=ran, torch=torch, binding=lambda: [c for c in ran if any("py_paged" in x for x in c)])


@pytest.mark.parametrize("version,cuda", [(None, True), ("2.11.0+cpu", False)])
def test_library_builds_without_torch(bench, version, cuda):
    bench.torch.version, bench.torch.cuda = version, cuda
    assert not b.up_to_date()
    b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.EXT)
    assert len(bench.ran) == len(b.SOURCES) + 1 and bench.binding() == []
    assert not any("torch" in x for c in bench.ran for x in c)
    assert b.up_to_date()
    bench.ran.clear()
    b.build()
    assert bench.ran == []


def test_binding_follows_when_torch_comes(bench):
    bench.torch.version = None
    b.build()
    bench.ran.clear()
    bench.torch.version = "2.11.0+cu130"
    assert not b.up_to_date()
    b.build()
    assert len(bench.ran) == 2 and bench.binding() == bench.ran      # compiled and linked; the library as it was
    assert b.up_to_date()


def test_binding_of_another_torch_is_not_current(bench):
    b.build()
    assert b.up_to_date() and len(bench.binding()) == 2
    bench.ran.clear()
    bench.torch.version = "2.11.0+cu130"
    assert not b.up_to_date()
    b.build()
    assert len(bench.ran) == 2 and b.up_to_date()


def test_newer_sources_build_what_needs_them(bench, monkeypatch, tmp_path):
    b.build()
    bench.ran.clear()
    old = os.path.getmtime(b.EXT)
    os.utime(b.LIB, (1, 1))                      # older than every .cu
    b.build()
    assert len(bench.ran) == len(b.SOURCES) + 1 and os.path.getmtime(b.EXT) == old
    bench.ran.clear()
    os.utime(b.EXT, (1, 1))
    b.build()
    assert len(bench.ran) == 2 and bench.binding() == bench.ran


def test_forced_build_is_whole(bench):
    b.build()
    bench.ran.clear()
    b.build(force=True)
    assert len(bench.ran) == len(b.SOURCES) + 3
