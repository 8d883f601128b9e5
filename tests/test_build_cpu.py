"""The build's host logic with stand-ins for the compilers: the C library needs nvcc alone."""
import os
import subprocess
import sys

import pytest

from linear_attention_recurrence_05_b200 import build as b


@pytest.fixture
def tree(repo_tmp, monkeypatch):
    """The build writing to a scratch directory; the compilers leave an empty output each.  Returns the
    commands that were run."""
    for name, rel in (("LIB", "libgdn.so"), ("FAST", "_fast.so"), ("BUILD", "_build")):
        monkeypatch.setattr(b, name, os.path.join(repo_tmp, rel))
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    return runs


def test_library_is_built_without_pytorch(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not os.path.exists(b.FAST) and all(cmd[0] == b.NVCC for cmd in tree)


def test_library_is_built_before_the_host_path(tree, monkeypatch):
    ran = b.subprocess.run

    def run(cmd, **kw):
        return subprocess.CompletedProcess(cmd, 1, "", "no Python.h") if cmd[0] == "g++" else ran(cmd, **kw)

    monkeypatch.setattr(b.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="no Python.h"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.FAST)


def test_up_to_date_files_are_kept(tree):
    b.build()
    n = len(tree)
    b.build()
    assert n > 2 and len(tree) == n
    b.build(force=True)
    assert len(tree) == 2 * n
