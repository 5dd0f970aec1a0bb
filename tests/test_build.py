"""build.build() with a stand-in for the compiler: what is compiled again, and what is linked."""
import os
import stat

import pytest

from exact_tiled_attention_36_b200 import build as fbuild

FAKE = """#!/usr/bin/env python3
import sys
a = sys.argv[1:]
out = a[a.index("-o") + 1]
open({log!r}, "a").write(" ".join(a) + "\\n")
if "-c" in a:
    src = a[a.index("-c") + 1]
    open(a[a.index("-MF") + 1], "w").write(out + ": " + src + "\\n")
    open(out, "w").write(" ".join(x for x in a if x.startswith("-D")) + ";")
else:
    open(out, "w").write("".join(open(x).read() for x in a if x.endswith(".o")))
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    log, nvcc = tmp_path / "log", tmp_path / "nvcc"
    nvcc.write_text(FAKE.format(log=str(log)))
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    srcs = [tmp_path / f"{n}.cu" for n in "abc"]
    for i, s in enumerate(srcs):
        s.write_text("")
        os.utime(s, (1000 + i, 1000 + i))
    monkeypatch.setattr(fbuild, "NVCC", str(nvcc))
    monkeypatch.setattr(fbuild, "SRCS", [str(s) for s in srcs])
    monkeypatch.setattr(fbuild, "DEPS", [str(s) for s in srcs])
    monkeypatch.setattr(fbuild, "OBJ_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(fbuild, "LIB", str(tmp_path / "lib.so"))

    def run(edit=None, **kw):
        """The sources compiled by this build, and the flags of the objects in the library."""
        log.write_text("")
        if edit is not None:
            later = os.path.getmtime(fbuild.LIB) + 5  # a clock tick past every object
            os.utime(srcs[edit], (later, later))
        lib = fbuild.build(**kw)
        calls = log.read_text().splitlines()
        compiled = [os.path.basename(c.split("-c ")[1].split()[0])[0] for c in calls if " -c " in c]
        return "".join(sorted(compiled)), open(lib).read()

    return run


def test_builds_what_changed(tree):
    assert tree() == ("abc", ";;;")
    assert tree() == ("", ";;;")
    assert tree(edit=1)[0] == "b"
    assert tree(force=True) == ("abc", ";;;")


def test_objects_of_other_flags_are_not_linked(tree):
    assert tree() == ("abc", ";;;")
    assert tree(extra=["-DX"]) == ("abc", "-DX;-DX;-DX;")
    assert tree(edit=0) == ("a", ";;;")  # b and c as the plain build left them
    assert tree(extra=["-DX"]) == ("abc", "-DX;-DX;-DX;")  # again, for what the compiler prints


def test_a_library_of_other_flags_is_linked_anew(tree):
    tree(extra=["-DX"])
    assert tree() == ("abc", ";;;")
    tree(extra=["-DX"])
    assert tree() == ("", ";;;")


def test_another_compiler(tree, tmp_path, monkeypatch):
    tree()
    other = tmp_path / "nvcc2"
    other.write_text((tmp_path / "nvcc").read_text())
    other.chmod(0o755)
    monkeypatch.setattr(fbuild, "NVCC", str(other))
    assert tree() == ("abc", ";;;")
