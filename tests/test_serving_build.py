"""Building the library and the Python module of the serving calls (no GPU)."""

import os
import sys

import pytest

from mxfp4_w4a4_post_block_b200 import build


@pytest.fixture
def built():
    build.build()
    yield
    build.build()


def test_library_builds_without_torch(built, monkeypatch, capsys):
    """libbatq does not use torch: where it is not installed the library is built, and the module left out."""
    monkeypatch.setitem(sys.modules, "torch", None)  # an import of torch raises ImportError
    assert build.build() == build.LIB
    assert build._build_serving(False) is False
    assert "torch is not installed" in capsys.readouterr().err


def test_module_is_built_again_for_another_torch(built, monkeypatch):
    import torch
    before = os.stat(build.SERVING).st_mtime_ns
    build.build()
    assert os.stat(build.SERVING).st_mtime_ns == before
    monkeypatch.setattr(torch, "__version__", "0.0")
    build.build()
    assert os.stat(build.SERVING).st_mtime_ns != before
