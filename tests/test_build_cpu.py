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


@pytest.mark.parametrize("how", ["missing", "another"])
def test_calls_without_a_fitting_host_path_go_through_python(how, monkeypatch):
    """... with one warning, and with the Python way's own refusals."""
    import torch
    import linear_attention_recurrence_05_b200 as gdn
    from linear_attention_recurrence_05_b200 import _fast
    monkeypatch.setattr(gdn, "_calls", None)
    if how == "another":
        monkeypatch.setattr(_fast, "built_for", "PyTorch 0.0.0")
    else:
        monkeypatch.delattr(gdn, "_fast")
        monkeypatch.setitem(sys.modules, gdn.__name__ + "._fast", None)
    q, w, pos = torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16), torch.ones(128), torch.zeros(1, dtype=torch.int32)
    with pytest.warns(RuntimeWarning, match="_fast.so"), pytest.raises(TypeError, match="CUDA"):
        gdn.qsa_norm_rope(q, w, pos)
    kc, tab, blocks = torch.zeros(2, 4, 8, 128, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32), pos.view(1, 1, 1)
    with pytest.raises(TypeError, match="CUDA"):
        gdn.qsa_kv_append(q, q, w, pos, tab, kc, kc)
    with pytest.raises(TypeError, match="CUDA"):
        gdn.qsa_attention(q[:, :1].contiguous(), blocks, pos, tab, kc, kc)
    assert gdn._calls is gdn._NoCalls
