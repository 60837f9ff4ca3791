"""The library is built where its Python modules cannot be (no GPU, nothing compiled)."""
import os
import subprocess
import types

import pytest

from csr_spmm_gb300 import build as b


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """Build outputs in a folder of the test's; compilers that only write their output."""
    for name, value in (("LIB_DIR", tmp_path), ("OBJ_DIR", tmp_path / "obj"),
                        ("LIB", tmp_path / "libcsrspmm.so")):
        monkeypatch.setattr(b, name, str(value))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    return tmp_path, ran


def test_a_module_that_fails_is_reported_with_the_library_in_place(elsewhere, monkeypatch):
    tmp, _ = elsewhere

    def fails(force=False):
        raise RuntimeError("g++ failed on lm_calls.cpp")

    monkeypatch.setattr(b, "_lm_calls", fails)
    for _ in range(2):                       # built, then found up to date
        with pytest.raises(RuntimeError, match="lm_calls"):
            b.build(out=b.LIB)
        assert (tmp / "libcsrspmm.so").exists() and (tmp / "libcsrspmm.so.sha256").exists()


def test_without_python_headers_the_modules_are_left_out(elsewhere, monkeypatch, capsys):
    tmp, _ = elsewhere
    paths = {**b.sysconfig.get_paths(), "include": str(tmp / "none")}
    monkeypatch.setattr(b.sysconfig, "get_paths", lambda: paths)
    assert b.build(out=b.LIB) == str(tmp / "libcsrspmm.so")
    assert not (tmp / "_lm_calls.so").exists() and not (tmp / "_torch_outputs.so").exists()
    assert "no Python.h" in capsys.readouterr().err


def test_without_torch_for_cuda_its_module_is_left_out(elsewhere, monkeypatch, capsys):
    tmp, _ = elsewhere
    (tmp / "torch" / "lib").mkdir(parents=True)
    spec = types.SimpleNamespace(submodule_search_locations=[str(tmp / "torch")])
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: spec)
    assert b.build(out=b.LIB) == str(tmp / "libcsrspmm.so")
    assert (tmp / "_lm_calls.so").exists() and not (tmp / "_torch_outputs.so").exists()
    assert "without CUDA" in capsys.readouterr().err
    assert not os.path.exists(os.path.join(str(tmp), "_torch_outputs.so.sha256"))
