"""The build on machines that lack what only the binding's compiled calls need: the library is built all the same."""
import os
import sys

import pytest

from memory_bound_weight_gb300 import build as mbuild


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The compiled calls built to another place, with the compiler of the library known by its path."""
    mbuild.build()
    monkeypatch.setattr(mbuild, "FAST", str(tmp_path / "_fast.so"))
    monkeypatch.setenv("NVCC", mbuild._nvcc())
    return tmp_path


def test_without_pytorch_the_library_is_built(elsewhere, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # its import raises ImportError
    assert mbuild.build() == mbuild.LIB and os.path.exists(mbuild.LIB)
    assert not os.path.exists(mbuild.FAST)
    assert "marshalled in Python" in capsys.readouterr().err


def test_without_a_host_compiler_on_the_path_the_library_is_kept(elsewhere, monkeypatch, capsys):
    pytest.importorskip("torch")
    monkeypatch.setenv("PATH", str(elsewhere))
    assert mbuild.build() == mbuild.LIB and os.path.exists(mbuild.LIB)
    assert not os.path.exists(mbuild.FAST)
    assert "marshalled in Python" in capsys.readouterr().err


def test_compiled_calls_older_than_their_source_do_not_stay(elsewhere, monkeypatch):
    with open(mbuild.FAST, "w"):
        pass
    os.utime(mbuild.FAST, (0, 0))
    monkeypatch.setitem(sys.modules, "torch", None)
    mbuild.build()
    assert not os.path.exists(mbuild.FAST)
