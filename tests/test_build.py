"""The in-tree build, with scripts in the place of the compilers: what is compiled, and when."""
import os
import stat
import sys

import pytest

from bit_expert_ffn_moe_gb300 import _build

TOOL = """#!/bin/sh
echo "$0 $@" >> "%s"
out=""
while [ $# -gt 0 ]; do if [ "$1" = "-o" ]; then out="$2"; fi; shift; done
%s
"""


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """A build folder of its own; tool(name, body): what nvcc or g++ does after it has noted its call in the log."""
    log = tmp_path / "log"
    log.write_text("")

    def tool(name, body='echo made > "$out"'):
        path = tmp_path / "bin" / name
        path.parent.mkdir(exist_ok=True)
        path.write_text(TOOL % (log, body))
        path.chmod(path.stat().st_mode | stat.S_IXUSR)
    tool("nvcc")
    tool("g++")
    monkeypatch.setenv("CUDA_HOME", str(tmp_path))
    monkeypatch.setenv("PATH", str(tmp_path / "bin") + os.pathsep + os.environ["PATH"])
    for name, file in (("BUILD", ""), ("LIB", "libmoe_gb300.so"), ("TORCH_OPS", "moe_torch_ops.so")):
        monkeypatch.setattr(_build, name, str(tmp_path / "out" / file) if file else str(tmp_path / "out"))

    def calls():
        lines = log.read_text().splitlines()
        log.write_text("")
        return sum("nvcc" in line.split()[0] for line in lines), sum("g++" in line.split()[0] for line in lines)
    return tool, calls


def test_the_library_needs_no_torch(tools, monkeypatch):
    _, calls = tools
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch fails
    assert _build.build() == _build.LIB
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.TORCH_OPS)
    assert calls() == (len(_build.sources()) + 1, 0)
    _build.build()
    assert calls() == (0, 0)


def test_a_module_that_does_not_compile_leaves_the_library(tools):
    tool, calls = tools
    tool("g++", "exit 1")
    with pytest.raises(RuntimeError, match="torch_ops.cpp"):
        _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.TORCH_OPS)
    calls()
    _build.build(torch_ops=False)
    assert calls() == (0, 0)
    tool("g++")
    _build.build()
    assert calls() == (0, 2) and os.path.exists(_build.TORCH_OPS)


def test_another_torch_rebuilds_the_module_alone(tools, monkeypatch):
    _, calls = tools
    _build.build()
    assert calls() == (len(_build.sources()) + 1, 2)
    _build.build()
    assert calls() == (0, 0)
    monkeypatch.setattr(_build, "_torch_id", lambda: "another")
    _build.build()
    assert calls() == (0, 2)
    _build.build()
    assert calls() == (0, 0)
