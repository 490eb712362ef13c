"""The build in a folder of its own, from one small source: the library needs
no torch, and a binding that does not build leaves it there."""
import ctypes
import os

import pytest

from roofline_gb300 import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    src = tmp_path / "one.cu"
    src.write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    out = tmp_path / "out"
    monkeypatch.setattr(build, "BUILD", str(out))
    monkeypatch.setattr(build, "LIB", str(out / "libone.so"))
    monkeypatch.setattr(build, "BINDING", str(out / "_one.so"))
    monkeypatch.setattr(build, "_sources", lambda: [str(src)])
    return src


def _one():
    return ctypes.CDLL(build.LIB).one()


def test_library_without_torch(small, monkeypatch):
    real = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else real(name, *a))
    assert build.build() == build.LIB
    assert _one() == 1 and not os.path.exists(build.BINDING)
    # and it is up to date without one
    monkeypatch.setattr(build, "_compile", lambda *a: pytest.fail("compiled again"))
    assert build.build() == build.LIB


def test_library_when_the_binding_fails(small, monkeypatch):
    pytest.importorskip("torch")

    def fails(log_dir):
        raise RuntimeError("no headers")
    monkeypatch.setattr(build, "_compile_binding", fails)
    with pytest.raises(RuntimeError, match="no headers"):
        build.build()
    assert _one() == 1
    # the next build tries the binding again, and the library no more
    monkeypatch.setattr(build, "_compile", lambda *a: pytest.fail("compiled again"))
    with pytest.raises(RuntimeError, match="no headers"):
        build.build()


def test_stale_by_any_source(tmp_path):
    out, dep = tmp_path / "out", tmp_path / "dep"
    dep.write_text("")
    assert build._stale(str(out), [str(dep)])
    out.write_text("")
    os.utime(dep, (1, 1))
    assert not build._stale(str(out), [str(dep)])
    os.utime(out, (0, 0))
    assert build._stale(str(out), [str(dep)])
