"""The build's two products: libes.so stands by itself, es_torch.so follows the
installed PyTorch.  A library of one function in a folder of its own."""
import ctypes
import os
import subprocess
import sys

import pytest

from element_scan_recurrences_gb300 import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    at = tmp_path / "_build"
    for name, value in (("BUILD", at), ("LIB", at / "libes.so"), ("TORCH_LIB", at / "es_torch.so"),
                        ("TORCH_STAMP", at / "es_torch.so.built_for"), ("GEN", at / "gen")):
        monkeypatch.setattr(build, name, str(value))
    monkeypatch.setattr(build, "_sources", lambda: [str(src)])
    return src


def linked():
    return ctypes.CDLL(build.LIB).one()


def stand_in(monkeypatch, code=0, calls=None):
    """A compilation of es_torch.cpp that takes no time."""
    def compile_torch(obj):
        if calls is not None:
            calls.append(obj)
        return "es_torch.cpp", subprocess.run([sys.executable, "-c", "raise SystemExit(%d)" % code], capture_output=True, text=True)

    def link_torch(obj):
        for path, text in ((build.TORCH_LIB, ""), (build.TORCH_STAMP, build._installed_torch())):
            with open(path, "w") as f:
                f.write(text)
    monkeypatch.setattr(build, "_compile_torch", compile_torch)
    monkeypatch.setattr(build, "_link_torch", link_torch)


def test_the_library_is_there_when_the_module_fails(small, monkeypatch):
    stand_in(monkeypatch, code=1)
    with pytest.raises(RuntimeError, match="es_torch"):
        build.build()
    assert linked() == 1 and not build.up_to_date()

    def broken(obj):
        raise ImportError("torch is broken")
    monkeypatch.setattr(build, "_compile_torch", broken)
    os.remove(build.LIB)
    with pytest.raises(ImportError):
        build.build()
    assert os.path.exists(build.LIB)


def test_without_pytorch_the_library_alone(small, monkeypatch):
    monkeypatch.setattr(build, "_installed_torch", lambda: None)
    monkeypatch.setattr(build, "_compile_torch", lambda obj: pytest.fail("there is no PyTorch to compile against"))
    assert not build.up_to_date()
    build.build()
    assert linked() == 1 and build.up_to_date() and not os.path.exists(build.TORCH_LIB)
    build.build(force=True)


def test_another_pytorch_builds_the_module_again_and_only_that(small, monkeypatch):
    calls = []
    stand_in(monkeypatch, calls=calls)
    build.build()
    assert len(calls) == 1 and build.up_to_date()
    build.build()
    assert len(calls) == 1
    t = os.path.getmtime(build.LIB)
    monkeypatch.setattr(build, "_installed_torch", lambda: "torch 99.0, another")
    assert not build.up_to_date()
    build.build()
    assert len(calls) == 2 and build.up_to_date() and os.path.getmtime(build.LIB) == t
