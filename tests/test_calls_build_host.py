"""The extension that reads the expert layer's arguments is built and loaded apart from libctr (CPU only)."""
import os
import shutil
import sysconfig

import pytest

from sparse_embeddings_feature_gb300 import build as B
from sparse_embeddings_feature_gb300 import ctr


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A build directory with libctr as it is built now, and no extension."""
    B.build()
    for name in ("libctr.so", "fingerprint"):
        shutil.copy(os.path.join(B.OUT_DIR, name), tmp_path / name)
    monkeypatch.setattr(B, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libctr.so"))
    monkeypatch.setattr(B, "CALLS", str(tmp_path / "ctr_calls.so"))
    monkeypatch.setattr(ctr, "_calls", None)
    monkeypatch.setenv("CTR_NVCC_EXTRA", os.environ.get("CTR_NVCC_EXTRA", ""))
    return tmp_path


@pytest.mark.parametrize("command", [["false"], ["/no/such/compiler"]])
def test_libctr_does_without_the_extension(place, monkeypatch, command):
    runs = []
    monkeypatch.setattr(B, "_calls_command", lambda out: runs.append(out) or command)
    with pytest.warns(RuntimeWarning, match="calls.cpp"):
        assert B.build() == B.LIB
    n = len([r for r in runs if r])
    assert B.build() == B.LIB and B.build_calls() is None     # known: not tried or said again
    assert len([r for r in runs if r]) == n
    assert ctr._usual().expert_route(1, 2) is None
    assert ctr.ctr_expert_workspace_size() == 256             # the library itself is there
    with pytest.raises(ValueError):                            # and the general binding serves the call
        ctr.ctr_expert_dispatch(None, None, None, None, None)


def test_an_extension_that_cannot_be_loaded(place):
    assert B.build_calls() == B.CALLS
    with open(B.CALLS, "wb") as f:
        f.write(b"not a library")
    with pytest.warns(RuntimeWarning, match="cannot be loaded"):
        assert ctr._usual().expert_route(1, 2) is None


def test_the_extension_is_for_this_python(place, monkeypatch):
    assert B.build_calls() == B.CALLS
    made = os.stat(B.CALLS).st_mtime_ns
    assert B.build_calls() == B.CALLS and os.stat(B.CALLS).st_mtime_ns == made
    mine = B._calls_fingerprint()
    var = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-399-other" if n == "SOABI" else var(n))
    assert B._calls_fingerprint() != mine
    monkeypatch.undo()
    monkeypatch.setenv("CXX", "another-compiler")
    assert B._calls_fingerprint() != mine
    monkeypatch.undo()
    monkeypatch.setattr("sys.version", "4.0")
    assert B._calls_fingerprint() != mine
