"""The build where what the binding alone needs is missing: the library is there all the same."""
import os
import shutil

import pytest

import bit_nf4_quantized_09_amd as nf4
from bit_nf4_quantized_09_amd import build, decoder


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A build of one source into a folder of its own, in which a binding of an earlier build lies."""
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "PROBE_LIB", str(tmp_path / "probe.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setattr(build, "SOURCES", ["rope.hip"])
    (tmp_path / "binding.so").write_bytes(b"of another build")


@pytest.mark.skipif(shutil.which(build.HIPCC) is None, reason="needs hipcc")
def test_library_without_a_compiler_for_the_binding(small, monkeypatch):
    monkeypatch.setenv("CXX", "no-such-compiler")
    with pytest.warns(UserWarning, match="no-such-compiler"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_binding_without_python_headers(small, monkeypatch, tmp_path):
    import sysconfig

    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    with pytest.warns(UserWarning, match="Python.h"):
        build._build_binding(False)
    assert not os.path.exists(build.BINDING)


@pytest.mark.skipif(shutil.which("false") is None, reason="needs false")
def test_a_binding_that_does_not_compile_fails_the_build(small, monkeypatch):
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(RuntimeError):
        build._build_binding(False)


def test_calls_say_that_the_binding_is_not_built(monkeypatch, tmp_path):
    monkeypatch.setattr(decoder, "_bound", None)
    monkeypatch.setattr(decoder, "binding_path", lambda: str(tmp_path / "binding.so"))
    with pytest.raises(nf4.NF4Error, match="not built"):
        nf4.rope_fwd(nf4.rope_plan(8, device="cpu"), None, None)
