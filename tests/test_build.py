"""What the build makes when, with small stand-ins for the sources: the C library never depends on PyTorch or g++."""
import importlib.util

import pytest

from quantized_matmul_speculative_gb300 import build

UNIT = 'extern "C" int qmm_stand_in(int x) { return x + 1; }\n'


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build's paths in a folder of their own: one small CUDA unit, and a module source that g++ takes at once."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "unit.cu").write_text(UNIT)
    (csrc / "qmm_torch.cpp").write_text("int qmm_nothing;\n")
    objects = tmp_path / "objects"
    for name, value in (("CSRC", csrc), ("PKG", tmp_path), ("BUILD", objects), ("LIBRARY", tmp_path / "libqmm.so"),
                        ("MODULE", tmp_path / "_qmm_torch.so"), ("MODULE_MADE_FOR", objects / "qmm_torch.for")):
        monkeypatch.setattr(build, name, value, raising=False)
    monkeypatch.setattr(build, "units", lambda: [(csrc / "unit.cu", objects / "unit.o", [])])
    return tmp_path


def without_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setitem(__import__("sys").modules, "torch", None)  # an import of it fails


def test_without_torch(tree, monkeypatch):
    """The library alone, and nothing to do the second time."""
    without_torch(monkeypatch)
    assert build.build() == build.LIBRARY and build.LIBRARY.exists() and not build.MODULE.exists()
    assert build.up_to_date()
    made = build.LIBRARY.stat().st_mtime_ns
    build.build()
    assert build.LIBRARY.stat().st_mtime_ns == made


def test_module_that_does_not_compile(tree):
    """The failure is loud, and the library is there all the same."""
    (build.CSRC / "qmm_torch.cpp").write_text("#error no\n")
    with pytest.raises(RuntimeError, match="qmm_torch"):
        build.build()
    assert build.LIBRARY.exists() and not build.MODULE.exists() and not build.up_to_date()


def test_without_a_host_compiler_for_the_module(tree, monkeypatch):
    run = build.subprocess.run

    def no_gpp(cmd, *a, **kw):
        if cmd[0] == "g++":
            raise FileNotFoundError("g++")
        return run(cmd, *a, **kw)

    monkeypatch.setattr(build.subprocess, "run", no_gpp)
    with pytest.raises((RuntimeError, FileNotFoundError), match=r"g\+\+"):
        build.build()
    assert build.LIBRARY.exists()


def test_module_of_another_torch_is_made_again(tree, monkeypatch):
    """A module is for one version of PyTorch and of Python; the library is left as it is."""
    pytest.importorskip("torch")
    build.build()
    assert build.up_to_date()
    library, module = build.LIBRARY.stat().st_mtime_ns, build.MODULE.stat().st_mtime_ns
    monkeypatch.setattr(build, "module_target", lambda: "another one")
    assert not build.up_to_date()
    build.build()
    assert build.up_to_date()
    assert build.MODULE.stat().st_mtime_ns > module and build.LIBRARY.stat().st_mtime_ns == library
