"""The library's build needs hipcc alone; the binding's native half is a step
of its own and carries the ABI it was built for in its name."""
import importlib.util
import os
import subprocess
import sysconfig

import pytest

from fp8_prefill_gemm_amd import build as b


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """The compilers' command lines, each output an empty file; the library in tmp_path."""
    seen = []

    def run(cmd, **kw):
        seen.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b, "LIB_PATH", str(tmp_path / b.LIB_NAME))
    return seen


@pytest.fixture
def no_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_library_without_torch(commands, no_torch):
    assert b.build() == b.LIB_PATH and os.path.exists(b.LIB_PATH)
    assert len(commands) == 1 and "hipcc" in commands[0][0] and not any("torch/" in a or "python" in a for a in commands[0])


def test_both_steps_where_torch_is(commands, monkeypatch, tmp_path):
    pytest.importorskip("torch")
    monkeypatch.setattr(b, "PKG_DIR", str(tmp_path))
    made = b.build_all()
    assert made == [b.LIB_PATH, b.native_path()] and all(os.path.exists(p) for p in made)
    assert [os.path.basename(c[0]) for c in commands] == ["hipcc", "g++"]


def test_both_steps_without_torch(commands, no_torch, capsys):
    """The library is built all the same, and what is left out is said."""
    assert b.build_all() == [b.LIB_PATH]
    assert "torch" in capsys.readouterr().err


def test_native_step_without_torch(commands, no_torch):
    with pytest.raises(RuntimeError, match="torch"):
        b.build_native()
    assert not commands


def test_native_name_has_the_abi(monkeypatch):
    torch = pytest.importorskip("torch")
    name = os.path.basename(b.native_path())
    assert name.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and torch.__version__ in name
    monkeypatch.setattr(b.importlib.metadata, "version", lambda p: "9.9.9")
    assert os.path.basename(b.native_path()) != name
