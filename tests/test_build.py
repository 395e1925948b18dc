"""The build's order, with stand-ins for the compilers: what the C library needs
does not hang on the Python binding."""
import os
import subprocess

import pytest

from speculative_decoding_verification_19_gb300 import build as b


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    """Paths of a build of its own, and compilers that write a file each, or fail
    for the commands that `broken` picks."""
    state = dict(broken=lambda cmd: False, seen=[])
    for name, path in (("BUILD", "_build"), ("LIB", "lib.so"), ("BIND", "bind.so")):
        monkeypatch.setattr(b, name, str(tmp_path / path))
    monkeypatch.setattr(b, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")

    def run(cmd, **kw):
        state["seen"].append(cmd)
        bad = state["broken"](cmd)
        if not bad:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write(str(len(state["seen"])))
        return subprocess.CompletedProcess(cmd, int(bad), "", "no Python.h" if bad else "")

    monkeypatch.setattr(b.subprocess, "run", run)
    return state


def binding(cmd):
    return any("binding" in c for c in cmd)


def test_everything_is_built_once(compilers):
    b.build()
    assert os.path.exists(b.LIB) and os.path.exists(b.BIND)
    n = len(compilers["seen"])
    b.build()
    assert len(compilers["seen"]) == n


@pytest.mark.parametrize("first", [False, True])
def test_the_library_without_the_binding(compilers, first):
    if first:  # an older build's binding does not outlive its library
        b.build()
    compilers["broken"] = binding
    with pytest.raises(RuntimeError, match="binding"):
        b.build(force=True)
    assert os.path.exists(b.LIB) and not os.path.exists(b.BIND)
    compilers["broken"] = lambda cmd: False
    b.build()  # nothing says that the failed build was whole
    assert os.path.exists(b.BIND)
