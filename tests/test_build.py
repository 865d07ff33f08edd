"""The incremental build: which objects are kept (with a stand-in for the compiler)."""
import os
import stat

import pytest

from sliding_window_global_b200 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source tree of two files, and a compiler that writes its command line to its output."""
    csrc, include = tmp_path / "csrc", tmp_path / "include"
    csrc.mkdir()
    include.mkdir()
    for name in ("csrc/a.cu", "csrc/b.cu", "csrc/h.cuh", "include/swa.h"):
        (tmp_path / name).write_text("")
        os.utime(tmp_path / name, (1, 1))
    nvcc = tmp_path / "nvcc"
    # an object holds its flags; the library holds its objects
    nvcc.write_text('#!/bin/sh\nout= ; prev=\nfor a in "$@"; do [ "$prev" = -o ] && out=$a; prev=$a; done\n'
                    'case "$out" in *.so.tmp) for a in "$@"; do case "$a" in *.o) cat "$a";; esac; done > "$out";;\n'
                    '*) echo "$@" > "$out";; esac\n')
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build, "CSRC", str(csrc))
    monkeypatch.setattr(build, "INCLUDE", str(include))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libswa.so"))
    monkeypatch.setattr(build, "NVCC", str(nvcc))
    return tmp_path


def _compiled(tree):
    return (tree / "libswa.so").read_text().splitlines()


def test_objects_of_other_flags_are_not_linked(tree):
    """A build with flags of its own between two plain ones leaves nothing in the second."""
    build.build()
    plain = _compiled(tree)
    assert len(plain) == 2 and not any("-G" in line for line in plain)
    build.build(force=True, extra=["-G"])
    assert all("-G" in line.split() for line in _compiled(tree))
    late = os.path.getmtime(tree / "libswa.so") + 5
    os.utime(tree / "csrc" / "a.cu", (late, late))                   # one source changes
    build.build()
    assert not any("-G" in line.split() for line in _compiled(tree))


def test_only_what_changed_is_compiled(tree):
    build.build()
    objs = [os.path.join(d, f) for d, _, files in os.walk(tree / "_build") for f in files]
    assert len(objs) == 2
    before = {o: os.path.getmtime(o) for o in objs}
    build.build()
    assert before == {o: os.path.getmtime(o) for o in objs}
    late = max(before.values()) + 5
    os.utime(tree / "csrc" / "b.cu", (late, late))
    build.build()
    changed = [os.path.basename(o) for o in objs if os.path.getmtime(o) != before[o]]
    assert changed == ["b.cu.o"]
    os.utime(tree / "csrc" / "h.cuh", (late + 5, late + 5))
    build.build()
    assert len(_compiled(tree)) == 2
