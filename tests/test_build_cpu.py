"""The build's host logic with stand-ins for the compilers: the C library needs nvcc alone, and the Python
package's host path is built for one PyTorch and Python."""
import os
import subprocess
import sys

import pytest

from linear_attention_recurrence_05_b200 import build as b


@pytest.fixture
def tree(repo_tmp, monkeypatch):
    """The build writing to a scratch directory; the compilers leave an empty output each.  Returns the
    commands that were run."""
    for name, rel in (("LIB", "libgdn.so"), ("FAST", "_fast.so"), ("BUILD", "_build"), ("FAST_KEY", "_build/_fast.key")):
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


def test_host_path_is_built_again_for_another_pytorch(tree, monkeypatch):
    import torch
    b.build()
    del tree[:]
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    b.build()
    assert [cmd[0] for cmd in tree] == ["g++"] and any("PyTorch 0.0.0" in a for a in tree[0])
    b.build()
    assert len(tree) == 1
    os.remove(b.FAST_KEY)                                # built for nobody knows what
    b.build()
    assert len(tree) == 2


def test_host_path_says_what_it_was_built_for():
    from linear_attention_recurrence_05_b200 import _fast
    assert _fast.built_for == b.fast_key()


def test_host_path_of_another_pytorch_is_not_called(monkeypatch):
    import linear_attention_recurrence_05_b200 as gdn
    from linear_attention_recurrence_05_b200 import _fast
    monkeypatch.setattr(gdn, "_calls", None)
    monkeypatch.setattr(_fast, "built_for", "PyTorch 0.0.0")
    with pytest.raises(RuntimeError, match="_fast.so"):
        gdn._load_calls()
    assert gdn._calls is None
