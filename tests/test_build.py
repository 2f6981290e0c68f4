"""What build() does without torch and with a binding that does not compile (on sources of its own)."""
import ctypes as C
import sys

import pytest


@pytest.fixture()
def build(tmp_path, monkeypatch):
    from streaming_selection_primitive_gb300 import build as b
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "answer.cpp").write_text('extern "C" int answer() { return 42; }\n')
    (src / "binding.cpp").write_text("this does not compile\n")
    for name, value in {"CSRC": src, "BUILD": tmp_path / "_build", "LIBDIR": tmp_path / "lib", "LIB": tmp_path / "lib" / "libprofk.so",
                        "BINDING_SOURCE": src / "binding.cpp", "SOURCES": ["answer.cpp"]}.items():
        monkeypatch.setattr(b, name, value)
    return b


def test_without_torch_the_library_is_built(build, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch: ModuleNotFoundError
    lib = build.build()
    assert C.CDLL(str(lib)).answer() == 42
    assert [p.name for p in build.LIBDIR.iterdir()] == ["libprofk.so"]
    before = lib.stat().st_mtime_ns
    assert build.build() == lib and lib.stat().st_mtime_ns == before  # nothing is stale


def test_a_failing_binding_raises_after_the_library_is_linked(build):
    pytest.importorskip("torch")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        build.build()
    assert C.CDLL(str(build.LIB)).answer() == 42
    with pytest.raises(RuntimeError):  # and again: what failed is not taken for done
        build.build()


def test_a_failing_unit_raises(build):
    (build.CSRC / "answer.cpp").write_text("nor does this\n")
    with pytest.raises(RuntimeError, match="answer.cpp"):
        build.build()
    assert not build.LIB.exists()
