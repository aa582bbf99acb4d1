"""The build: the library alone where there is no torch, and the torch module
made anew for another torch. On one small translation unit, in a folder of
its own."""
import os
import sys

import pytest

from all_reduce_residual_gb300 import build


@pytest.fixture()
def small(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "SOURCES", ["arf_measure.cu"])
    for name, file in (("BUILD_DIR", "o"), ("LIB", "libarf.so"), ("TORCH_LIB", "_torch_ops.so")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    return tmp_path


def test_library_without_torch(monkeypatch, small):
    monkeypatch.setitem(sys.modules, "torch", None)  # importing it fails, as where it is not installed
    assert build.stale()
    build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.TORCH_LIB)
    assert not build.stale()


def test_module_follows_torch(monkeypatch, small):
    """The module of another torch, or of another interpreter, is out of date."""
    monkeypatch.setattr(build, "TORCH_STAMP", str(small / "stamp"))
    for name in ("libarf.so", "_torch_ops.so"):
        (small / name).write_text("")
    assert build.stale()  # made before it was noted what for
    (small / "stamp").write_text(build._torch_stamp())
    assert not build.stale()
    (small / "stamp").write_text(build._torch_stamp().replace(sys.version, "3.0"))
    assert build.stale()
    (small / "stamp").write_text(build._torch_stamp() + "# another")
    assert build.stale()
    monkeypatch.setitem(sys.modules, "torch", None)
    assert not build.stale()
