"""The compiled marshalling where it does not fit the PyTorch that runs: the Python functions make the calls."""
import os
import shutil
import warnings

import pytest

torch = pytest.importorskip("torch")

from memory_bound_weight_gb300 import _binding as B  # noqa: E402
from memory_bound_weight_gb300 import build as mbuild  # noqa: E402


@pytest.fixture
def unloaded(monkeypatch, tmp_path):
    """A binding that has not looked for its compiled calls, and looks for them in a folder of the test's."""
    mbuild.build()
    B.lib()
    monkeypatch.setattr(B, "LIB_PATH", str(tmp_path / "libmbw.so"))
    monkeypatch.setattr(B, "_fast", None)
    return str(tmp_path / "_fast.so")


def test_a_file_that_does_not_load_is_left_alone(unloaded):
    with open(unloaded, "w") as f:
        f.write("no library")
    with pytest.warns(RuntimeWarning, match="marshalled in Python"):
        B._load_fast()
    assert B._fast is False


def test_a_build_for_another_pytorch_is_left_alone(unloaded, monkeypatch):
    if not os.path.exists(mbuild.FAST):
        pytest.skip("not built here")
    shutil.copy(mbuild.FAST, unloaded)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    with pytest.warns(RuntimeWarning, match="built for"):
        B._load_fast()
    assert B._fast is False


def test_this_build_is_used(unloaded):
    if not os.path.exists(mbuild.FAST):
        pytest.skip("not built here")
    shutil.copy(mbuild.FAST, unloaded)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        B._load_fast()
    assert B._fast and B._fast.built_for.endswith(torch.__version__)


def test_no_file_is_no_cause_for_a_warning(unloaded):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        B._load_fast()
    assert B._fast is False


def test_another_pytorch_makes_the_file_stale(monkeypatch, tmp_path):
    mbuild.build()
    monkeypatch.setattr(mbuild, "FAST", str(tmp_path / "_fast.so"))
    monkeypatch.setattr(mbuild, "FAST_FOR", str(tmp_path / "_fast.for"))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(mbuild.FAST + ".tmp", "w"):
            pass
        return mbuild.subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(mbuild.subprocess, "run", run)
    for n in (1, 1):  # built once, then found
        mbuild._fast()
        assert len(ran) == n
    monkeypatch.setattr(mbuild, "_here", lambda: "another")
    mbuild._fast()
    assert len(ran) == 2
