"""The build: the library alone where there is no torch. On one small
translation unit, in a folder of its own."""
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
