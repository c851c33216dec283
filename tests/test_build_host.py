"""What build() makes anew, with the compilers replaced by one that writes its output file: no kernel is
compiled here. After a change of the C ABI no older Python module may stay beside the new library."""
import os
import subprocess
import types

import pytest

from token_level_sparse_hs2_b200 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source tree of one kernel, the module's source and the header, with everything built once."""
    here, inc = tmp_path / "pkg", tmp_path / "include"
    (here / "csrc").mkdir(parents=True)
    inc.mkdir()
    t = types.SimpleNamespace(kernel=here / "csrc" / "k.cu", module=here / "csrc" / "marshal.cpp", header=inc / "hs2.h",
                              lib=here / "libhs2.so", marshal=here / "_marshal.so", runs=[], broken=(), missing=(), clock=1_000_000_000)
    for f in (t.kernel, t.module, t.header):
        f.write_text("")
    for name, value in (("HERE", here), ("ROOT", tmp_path), ("CSRC", here / "csrc"), ("BUILD", here / "_build"), ("LIB", t.lib),
                        ("MARSHAL", t.marshal)):
        monkeypatch.setattr(B, name, str(value))

    def stamp(path):            # a file's time is the order of its making, whatever the clock's steps
        t.clock += 10
        os.utime(path, (t.clock, t.clock))

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        name = os.path.basename(out).split(".tmp")[0]
        t.runs.append(name)
        if os.path.basename(cmd[0]) in t.missing:
            raise FileNotFoundError(cmd[0])
        if name in t.broken:
            return subprocess.CompletedProcess(cmd, 1, "", "broken")
        with open(out, "w") as f:
            f.write(t.header.read_text())       # what it was made from
        stamp(out)
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def change(path, text):
        path.write_text(text)
        stamp(path)

    def build(broken=(), fails=False):
        t.runs.clear()
        t.broken = broken
        if fails:
            with pytest.raises((RuntimeError, OSError)):
                B.build()
        else:
            B.build()
        return set(t.runs)

    monkeypatch.setattr(B.subprocess, "run", run)
    monkeypatch.setattr(B, "nvcc", lambda: "nvcc")
    t.build, t.change = build, change
    for f in (t.kernel, t.module, t.header):
        stamp(f)
    assert build() == {"k.cu.o", "marshal.cpp.o", "libhs2.so", "_marshal.so"}
    return t


def test_nothing_changed_is_nothing_made(tree):
    assert tree.build() == set()


def test_a_changed_kernel_leaves_the_module(tree):
    tree.change(tree.kernel, "other")
    assert tree.build() == {"k.cu.o", "libhs2.so"}


@pytest.mark.parametrize("broken", ["k.cu.o", "libhs2.so", "_marshal.so", "marshal.cpp.o"])
def test_a_build_that_fails_leaves_no_older_module_behind_for_the_next(tree, broken):
    tree.change(tree.header, "new signature")
    tree.build(broken=(broken,), fails=True)
    tree.build()
    assert tree.lib.read_text() == tree.marshal.read_text() == "new signature"


@pytest.mark.parametrize("broken", ["_marshal.so", "marshal.cpp.o"])
def test_no_older_module_beside_a_new_library(tree, broken):
    tree.change(tree.header, "new signature")
    tree.build(broken=(broken,), fails=True)
    assert tree.lib.exists() and (tree.lib.read_text() == "" or not tree.marshal.exists())


def test_the_library_needs_no_torch(tree, monkeypatch):
    import sys
    tree.change(tree.header, "new signature")
    monkeypatch.setitem(sys.modules, "torch", None)                  # import torch raises ImportError
    assert tree.build() == {"k.cu.o", "libhs2.so"}
    assert tree.lib.read_text() == "new signature" and not tree.marshal.exists()
    monkeypatch.undo()


def test_the_library_needs_no_host_compiler_of_the_module(tree):
    tree.change(tree.header, "new signature")
    tree.missing = ("g++",)
    tree.build(fails=True)                                           # says so, with the library built
    assert tree.lib.read_text() == "new signature" and not tree.marshal.exists()
    tree.missing = ()
    assert tree.build() == {"marshal.cpp.o", "_marshal.so"}


def test_another_torch_is_a_new_module(tree, monkeypatch):
    import torch
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert tree.build() == {"marshal.cpp.o", "_marshal.so"}
    assert tree.build() == set()
