"""The build on a machine without torch, or without a host compiler: liblopt.so is linked all the same.  The compilers'
runs are replaced by empty files."""
import importlib.util
import os

import pytest

from learned_optimizer_step_amd import build as B


@pytest.fixture
def made(monkeypatch, tmp_path):
    """Builds into tmp_path; the commands that are run, by the base name of what they write."""
    for name, file in (("LIB", "liblopt.so"), ("LAYERS", "_layers.so"), ("MICROBENCH", "lopt_microbench")):
        monkeypatch.setattr(B, name, str(tmp_path / file))
    monkeypatch.setattr(B, "PKG", str(tmp_path))
    monkeypatch.setattr(B, "hipcc", lambda: "hipcc")
    ran = {}

    def run(cmd, verbose):
        if cmd[0] != "hipcc" and B.broken_compiler:
            raise RuntimeError("no host compiler")
        to = cmd[cmd.index("-o") + 1]
        ran[os.path.basename(to)] = cmd
        open(to, "w").close()

    monkeypatch.setattr(B, "_run", run)
    monkeypatch.setattr(B, "broken_compiler", False, raising=False)
    return ran


def test_everything(made, tmp_path):
    assert B.build(out=B.LIB) == B.LIB
    assert {"liblopt.so", "_layers.so", "lopt_microbench"} <= set(os.listdir(tmp_path))
    assert not any("lopt" in a for a in made["layers.so"][1:] if a.startswith("-l"))


def test_without_torch(made, tmp_path, monkeypatch, capsys):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert B.build(out=B.LIB) == B.LIB
    assert os.path.exists(tmp_path / "liblopt.so") and not os.path.exists(tmp_path / "_layers.so")
    assert "torch is not installed" in capsys.readouterr().err


def test_without_a_host_compiler(made, tmp_path, monkeypatch):
    monkeypatch.setattr(B, "broken_compiler", True)
    with pytest.raises(RuntimeError, match="no host compiler"):
        B.build(out=B.LIB)
    assert os.path.exists(tmp_path / "liblopt.so") and os.path.exists(tmp_path / "lopt_microbench")


def test_another_library_alone(made, tmp_path):
    B.build(out=str(tmp_path / "other.so"))
    assert os.path.exists(tmp_path / "other.so") and not os.path.exists(tmp_path / "_layers.so")
