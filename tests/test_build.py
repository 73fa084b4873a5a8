"""The build of the library from its translation units: what is compiled and linked when, with a stand-in compiler."""

import os
import subprocess
import time

import pytest

from masked_block_diffusion_b200 import build

FAKE = """#!/bin/bash
# compiles to a file that holds the source's text, links to one that holds the objects'
out= ; src=()
while [ $# -gt 0 ]; do
  case "$1" in
    -o) out="$2"; shift ;;
    *.cu|*.o) src+=("$1") ;;
  esac
  shift
done
echo "start $(basename "$out")" >> "$FAKE_LOG"
case "$(basename "$out")" in
  "$FAKE_SLOW"*) sleep 1 ;;
esac
case "$(basename "$out")" in
  "$FAKE_FAIL"*) exit 3 ;;
esac
cat "${src[@]}" > "$out"
echo "end $(basename "$out")" >> "$FAKE_LOG"
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    for d in ("csrc", "include"):
        (tmp_path / d).mkdir()
    (tmp_path / "include" / "dllm.h").write_text("")
    for n in ("a", "b"):
        (tmp_path / "csrc" / f"{n}.cu").write_text(f"{n}1 ")
    fake = tmp_path / "nvcc"
    fake.write_text(FAKE)
    fake.chmod(0o755)
    monkeypatch.setattr(build, "CSRC", str(tmp_path / "csrc"))
    monkeypatch.setattr(build, "INCLUDE", str(tmp_path / "include"))
    monkeypatch.setattr(build, "OBJ", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "UNITS", {"a": [], "b": []})
    monkeypatch.setattr(build, "nvcc", lambda: str(fake))
    monkeypatch.setenv("FAKE_LOG", str(tmp_path / "log"))
    monkeypatch.setenv("FAKE_FAIL", "none")
    monkeypatch.setenv("FAKE_SLOW", "none")
    return tmp_path


def settle(tree):
    """Everything built so far as old as its sources."""
    old = time.time() - 1000
    for p in tree.rglob("*"):
        if p.is_file():
            os.utime(p, (old, old))


def test_a_link_that_failed_is_made_up_for(tree, monkeypatch):
    build.build_dllm()
    assert (tree / "lib.so").read_text() == "a1 b1 "
    settle(tree)
    (tree / "csrc" / "a.cu").write_text("a2 ")
    monkeypatch.setenv("FAKE_FAIL", "lib.so")
    with pytest.raises(subprocess.CalledProcessError):
        build.build_dllm()
    assert (tree / "lib.so").read_text() == "a1 b1 "
    monkeypatch.setenv("FAKE_FAIL", "none")
    build.build_dllm()
    assert (tree / "lib.so").read_text() == "a2 b1 "


def test_a_unit_that_fails_does_not_leave_the_other_ones_compiler_behind(tree, monkeypatch):
    monkeypatch.setenv("FAKE_FAIL", "a.o")
    monkeypatch.setenv("FAKE_SLOW", "b.o")
    with pytest.raises(subprocess.CalledProcessError):
        build.build_dllm()
    assert "end b.o.tmp" in (tree / "log").read_text()
    assert (tree / "obj" / "b.o").exists() and not (tree / "lib.so").exists()
    monkeypatch.setenv("FAKE_FAIL", "none")
    build.build_dllm()
    assert (tree / "lib.so").read_text() == "a1 b1 "
    assert (tree / "log").read_text().count("start b.o") == 1            # what compiled is kept


def test_nothing_is_done_where_nothing_changed(tree):
    build.build_dllm()
    log = (tree / "log").read_text()
    build.build_dllm()
    assert (tree / "log").read_text() == log
    # a tree that got the library alone
    for n in ("a", "b"):
        (tree / "obj" / f"{n}.o").unlink()
    build.build_dllm()
    assert (tree / "log").read_text() == log
    # and one of whose sources changed since
    settle(tree)
    (tree / "csrc" / "b.cu").write_text("b2 ")
    build.build_dllm()
    assert (tree / "lib.so").read_text() == "a1 b2 "
