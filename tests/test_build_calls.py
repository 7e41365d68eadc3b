"""When the extension for calls from torch tensors is built again: for a newer source, and for
another torch or Python than the one it was built against."""
import os
import time

import pytest

from w4a8_quantized_gemm_02_b200 import build


@pytest.fixture
def made(monkeypatch, tmp_path):
    """build_calls with its files in tmp_path and a compiler that only writes its output;
    returns the number of builds so far."""
    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "version.py").write_text("__version__ = '1'")
    src = tmp_path / "src.cpp"
    src.write_text("")
    runs = []

    def compile_(cmd):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(str(len(runs)))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "calls.so"))
    monkeypatch.setattr(build, "CALLS_SRC", str(src))
    monkeypatch.setattr(build, "CALLS_STAMP", str(tmp_path / "_build" / "calls.txt"))
    monkeypatch.setattr(build, "INCLUDE", str(tmp_path))
    (tmp_path / "qoq.h").write_text("")
    monkeypatch.setattr(build, "_torch_dir", lambda: str(torch))
    monkeypatch.setattr(build.subprocess, "check_call", compile_)
    return lambda: (build.build_calls(), len(runs))[1]


def test_built_once(made):
    assert [made(), made(), made()] == [1, 1, 1]


def test_built_again_for_another_torch(made, tmp_path):
    assert made() == 1
    version = tmp_path / "torch" / "version.py"
    version.write_text("__version__ = '2'")
    os.utime(version, (1, 1))                # (installed files keep the times of their packaging)
    assert [made(), made()] == [2, 2]


def test_built_again_for_another_place_or_python(made, monkeypatch, tmp_path):
    assert made() == 1
    monkeypatch.setattr(build.sys, "version", "another")
    assert [made(), made()] == [2, 2]
    other = tmp_path / "other"
    other.mkdir()
    (other / "version.py").write_text("__version__ = '1'")
    monkeypatch.setattr(build, "_torch_dir", lambda: str(other))
    assert [made(), made()] == [3, 3]


def test_built_again_for_a_newer_source_or_without_a_stamp(made, tmp_path):
    assert made() == 1
    os.utime(tmp_path / "src.cpp", (time.time() + 60,) * 2)
    assert made() == 2
    os.utime(tmp_path / "src.cpp", (1, 1))
    os.remove(build.CALLS_STAMP)
    assert [made(), made()] == [3, 3]


def test_a_failed_build_leaves_no_stamp_of_success(made, monkeypatch, tmp_path):
    assert made() == 1
    (tmp_path / "torch" / "version.py").write_text("__version__ = '2'")

    def fail(cmd):
        raise RuntimeError("no compiler")
    monkeypatch.setattr(build.subprocess, "check_call", fail)
    for _ in range(2):
        with pytest.raises(RuntimeError):
            build.build_calls()
