"""What the build makes when: with compilers that only write down how they were called."""
import os
import stat
import sys

import pytest

from scaled_dot_product_forward_gb300 import _build

COMPILER = f"""#!{sys.executable}
import os, sys
name = os.path.basename(sys.argv[0])
out = sys.argv[sys.argv.index("-o") + 1]
with open(out, "w") as f:
    f.write(name)
with open(os.path.join(os.path.dirname(sys.argv[0]), "calls"), "a") as f:
    f.write(name + " " + os.path.basename(out) + chr(10))
"""


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    """An empty place to build into; the compilers' calls so far, forgotten by each look."""
    for name in ("nvcc", "g++"):
        path = tmp_path / name
        path.write_text(COMPILER)
        path.chmod(path.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("PATH", f"{tmp_path}{os.pathsep}{os.environ['PATH']}")
    monkeypatch.setattr(_build, "LIB_PATH", str(tmp_path / "out.so"))
    monkeypatch.setattr(_build, "BINDING_PATH", str(tmp_path / "binding.so"))

    def calls():
        path = tmp_path / "calls"
        done = path.read_text().split("\n")[:-1] if path.exists() else []
        path.unlink(missing_ok=True)
        return sorted(done)

    return calls


LIBRARY = sorted(["nvcc " + os.path.splitext(s)[0] + ".o" for s in _build.SOURCES] + ["nvcc " + _build.LIB_NAME])
BINDING = ["g++ binding.o", "g++ binding.so"]


def test_both_are_built_once(compilers):
    pytest.importorskip("torch")
    assert not _build.up_to_date()
    assert _build.build() == _build.LIB_PATH
    assert compilers() == sorted(LIBRARY + BINDING)
    assert os.path.exists(_build.LIB_PATH) and os.path.exists(_build.BINDING_PATH)
    assert _build.up_to_date() and _build.build() == _build.LIB_PATH and compilers() == []
    _build.build(force=True)
    assert compilers() == sorted(LIBRARY + BINDING)
    os.utime(_build.LIB_PATH, (0, 0))
    assert not _build.up_to_date()
    _build.build()
    assert compilers() == LIBRARY
    os.utime(_build.BINDING_PATH, (0, 0))
    assert not _build.up_to_date()
    _build.build()
    assert compilers() == BINDING and _build.up_to_date()


@pytest.mark.parametrize("force", [False, True])
def test_the_library_needs_no_torch(compilers, monkeypatch, force):
    with monkeypatch.context() as without:
        without.setitem(sys.modules, "torch", None)      # (an import of it fails)
        assert _build.build(force=force) == _build.LIB_PATH
        assert compilers() == LIBRARY
        assert os.path.exists(_build.LIB_PATH) and not os.path.exists(_build.BINDING_PATH)
        assert _build.up_to_date()
    pytest.importorskip("torch")
    # with torch, what is missing is made
    assert not _build.up_to_date()
    _build.build()
    assert compilers() == BINDING and _build.up_to_date()


def test_a_failed_compiler_is_named(compilers, tmp_path):
    (tmp_path / "nvcc").write_text("#!/bin/sh\necho no such thing; exit 3\n")
    with pytest.raises(RuntimeError, match="nvcc failed(.|\n)*no such thing"):
        _build.build()
    assert not os.path.exists(_build.LIB_PATH) and not os.path.exists(_build.BINDING_PATH)


@pytest.fixture
def torch():
    return pytest.importorskip("torch")


def test_a_binding_of_another_torch_is_built_again(compilers, torch, monkeypatch):
    _build.build()
    compilers()
    with monkeypatch.context() as other:
        other.setattr(torch, "__version__", "0.0.1+other")
        assert not _build.up_to_date()
        _build.build()
        assert compilers() == BINDING and _build.up_to_date()
    assert not _build.up_to_date()      # (made for that one now)
    _build.build()
    assert compilers() == BINDING and _build.up_to_date()
    # one that does not say what it was made for
    os.unlink(_build.binding_key_path())
    assert not _build.up_to_date()


def test_a_binding_of_another_torch_is_not_loaded(torch, monkeypatch):
    import scaled_dot_product_forward_gb300 as sdpa
    _build.build()
    monkeypatch.setattr(sdpa, "_native", None)
    with monkeypatch.context() as other:
        other.setattr(torch, "__version__", "0.0.1+other")
        with pytest.raises(ImportError, match="built for .*torch.*build it again"):
            sdpa.SdpaPagedCache(None, None)
        assert sdpa._native is None
    sdpa._need_torch()
    assert sdpa._native is not None
