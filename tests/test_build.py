"""What build_lib builds, and when (a stand-in for nvcc that writes its output file; no compiler is run)."""
import os
import stat

import pytest

from fp64_gemm_emulation_gb300 import build_lib


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source tree with one kernel file; calls: the stand-in's command lines."""
    src, log = tmp_path / "csrc", tmp_path / "calls"
    src.mkdir()
    (src / "a.cu").write_text("// a kernel\n")
    (src / "tensor_lists.cpp").write_text("// a module\n")
    fake = tmp_path / "nvcc"
    fake.write_text(f'#!/bin/sh\necho "$@" >> {log}\nwhile [ "$1" != -o ]; do shift; done\necho made > "$2"\n')
    fake.chmod(fake.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("NVCC", str(fake))
    for name, path in (("CSRC", src), ("INCLUDE", tmp_path), ("BUILD", tmp_path / "_build"), ("LIB", tmp_path / "libozaki.so"), ("LISTS", tmp_path / "_tensor_lists.so")):
        monkeypatch.setattr(build_lib, name, str(path))

    def calls():
        lines = log.read_text().splitlines() if log.exists() else []
        log.unlink(missing_ok=True)
        return ["link" if "-shared" in line.split() else "compile" for line in lines]

    return tmp_path, calls


def test_the_library_needs_no_helper(tree, monkeypatch, capsys):
    def fails(*_):
        raise RuntimeError("no torch here")

    monkeypatch.setattr(build_lib, "build_lists", fails)
    tmp, calls = tree
    assert build_lib.build() == str(tmp / "libozaki.so") and (tmp / "libozaki.so").exists()
    assert calls() == ["compile", "link"]
    assert "no torch here" in capsys.readouterr().err
    build_lib.build()
    assert calls() == []


def test_objects_newer_than_the_library_are_linked(tree, monkeypatch):
    monkeypatch.setattr(build_lib, "build_lists", lambda *_: "")
    tmp, calls = tree
    build_lib.build()
    calls()
    then = os.path.getmtime(tmp / "_build" / "a.o")
    os.utime(tmp / "libozaki.so", (then - 100, then - 100))  # as a build leaves it that ended before its link
    build_lib.build()
    assert calls() == ["link"]


def test_the_helper_is_built_anew_for_another_torch(tree, monkeypatch):
    import torch

    tmp, _ = tree
    (tmp / "bin").mkdir()
    fake = tmp / "bin" / "g++"
    fake.write_text((tmp / "nvcc").read_text().replace("calls", "gxx"))
    fake.chmod(fake.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("PATH", str(tmp / "bin"), prepend=os.pathsep)

    def built():
        build_lib.build_lists()
        log = tmp / "gxx"
        n = len(log.read_text().splitlines()) if log.exists() else 0
        log.unlink(missing_ok=True)
        return n

    assert [built(), built()] == [1, 0]
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert [built(), built()] == [1, 0]
    (tmp / "_build" / "tensor_lists.for").unlink()  # one that was built before this was kept
    assert [built(), built()] == [1, 0]


@pytest.mark.parametrize("there, says", [(True, "undefined symbol"), (False, "is missing")])
def test_a_helper_that_does_not_load_says_why(there, says, monkeypatch, tmp_path):
    import sys

    import fp64_gemm_emulation_gb300 as package
    from fp64_gemm_emulation_gb300 import ozaki as oz

    class Fails:
        def find_spec(self, name, *_):
            if name.endswith("_tensor_lists"):
                raise ImportError("undefined symbol: f")

    monkeypatch.setattr(oz, "_PKG", str(tmp_path))
    if there:
        (tmp_path / "_tensor_lists.so").write_text("")
    monkeypatch.delitem(sys.modules, "fp64_gemm_emulation_gb300._tensor_lists", raising=False)
    monkeypatch.delattr(package, "_tensor_lists", raising=False)
    monkeypatch.setattr(sys, "meta_path", [Fails(), *sys.meta_path])
    with pytest.raises(ImportError, match=says):
        oz._tensor_lists()
