"""Which sources a build compiles, with a compiler that only writes its output file."""
import os
import subprocess
import time

import pytest

from int4_linear_b200 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    old = time.time() - 1000
    for name in ("a.cu", "b.cu", "c.cuh"):
        (csrc / name).write_text("")
        os.utime(csrc / name, (old, old))
    monkeypatch.setattr(B, "HERE", str(tmp_path))
    monkeypatch.setattr(B, "CSRC", str(csrc))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "SOURCES", ["a.cu", "b.cu"])
    monkeypatch.setattr(B, "HEADERS", ["c.cuh"])
    compiled = []

    def run(cmd, check):
        if "-c" in cmd:
            src = os.path.basename(cmd[cmd.index("-c") + 1])
            if src in tree.broken:
                raise subprocess.CalledProcessError(1, cmd)
            compiled.append(src)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    monkeypatch.setattr(B.subprocess, "run", run)

    class Tree:
        broken = set()

        def build(self):
            compiled.clear()
            B.build()
            return sorted(compiled)

        def touch(self, name):
            later = time.time() + 1000
            os.utime(csrc / name, (later, later))

        def flags(self, *more):
            monkeypatch.setattr(B, "NVCC_FLAGS", [*B.NVCC_FLAGS, *more])
    tree = Tree()
    return tree


def test_what_changed_is_compiled(tree):
    assert tree.build() == ["a.cu", "b.cu"]
    assert tree.build() == []
    tree.touch("b.cu")
    assert tree.build() == ["b.cu"]


def test_other_flags_compile_everything(tree):
    """No library of objects of two sets of flags, whether or not a source changed as well."""
    tree.build()
    tree.flags("-DX")
    assert tree.build() == ["a.cu", "b.cu"]
    assert tree.build() == []
    tree.touch("a.cu")
    tree.flags("-DY")
    assert tree.build() == ["a.cu", "b.cu"]


def test_other_flags_after_a_build_that_failed(tree):
    """Objects of the new flags beside ones of the old are not taken for one set."""
    tree.build()
    tree.flags("-DX")
    tree.broken = {"b.cu"}
    with pytest.raises(subprocess.CalledProcessError):
        tree.build()
    tree.broken = set()
    assert tree.build() == ["a.cu", "b.cu"]


def test_objects_without_a_record_of_their_flags(tree):
    tree.build()
    os.remove(B._stamp())
    assert tree.build() == ["a.cu", "b.cu"]
