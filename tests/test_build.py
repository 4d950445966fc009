"""What is built, and what a part that cannot be built takes with it.  No compiler runs."""
import subprocess

import pytest

from rns_emulated_fp64_gb300 import binding
from rns_emulated_fp64_gb300 import build as b


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """A compiler that writes its output's name into it; everything goes to tmp_path."""
    def run(cmd, **kw):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "b"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "b" / "libos2.so"))
    monkeypatch.setattr(b, "BUILD_DEBUG", str(tmp_path / "d"))
    monkeypatch.setattr(b, "LIB_DEBUG", str(tmp_path / "d" / "libos2.so"))
    return tmp_path


def broken(force=False):
    raise RuntimeError("g++ failed")


def test_the_library_is_there_where_its_python_part_cannot_be_built(fake, monkeypatch):
    monkeypatch.setattr(b, "build_head", broken)
    for _ in range(2):                                   # built, and found up to date
        with pytest.raises(RuntimeError, match="g.. failed"):
            b.build()
        assert (fake / "b" / "libos2.so").read_text() == "built"
    assert b.build(debug=True) == str(fake / "d" / "libos2.so")
    assert (fake / "d" / "libos2.so").exists()


def test_loading_builds_the_library_alone(fake, monkeypatch):
    monkeypatch.setattr(b, "build_head", broken)
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setenv("OS2_LIB", "")
    with pytest.raises(OSError):                         # what the fake compiler wrote is no library
        binding.load()
    assert (fake / "b" / "libos2.so").exists()


def test_both_parts_are_built(fake, monkeypatch):
    seen = []
    monkeypatch.setattr(b, "build_head", lambda force=False: seen.append(force))
    assert b.build() == str(fake / "b" / "libos2.so") and b.build(force=True)
    assert seen == [False, True]
    with monkeypatch.context() as m:
        m.setattr(b.subprocess, "run", lambda cmd, **kw: subprocess.CompletedProcess(cmd, 1, "", "no"))
        with pytest.raises(RuntimeError, match="nvcc failed"):
            b.build(force=True)
