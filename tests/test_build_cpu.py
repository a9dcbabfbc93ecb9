"""The build's cache: what is made again when sources, flags or the compiler
change, and what a failed build leaves behind (with a compiler that only
writes down what it is asked)."""
import os
import subprocess
import textwrap
import time

import pytest

from gated_delta_rule_72_b200 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "gdn.h").write_text("")
    (csrc / "shared.cuh").write_text("")
    for name in ("a", "b"):
        (csrc / (name + ".cu")).write_text('#include "shared.cuh"\n' if name == "a" else "")
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(textwrap.dedent("""\
        #!/bin/sh
        dir=$(dirname "$0")
        if [ "$1" = --version ]; then cat "$dir/version"; exit 0; fi
        for out; do :; done
        echo "$@" >> "$dir/log"
        case "$*" in *a.cu*) [ -e "$dir/fail" ] && exit 1;; *b.cu*) [ -e "$dir/fail" ] && sleep 0.5;; esac
        echo "$@" > "$out"
        """))
    nvcc.chmod(0o755)
    (tmp_path / "version").write_text("one\n")
    monkeypatch.setenv("NVCC", str(nvcc))
    monkeypatch.setattr(build, "ROOT", str(tmp_path))
    monkeypatch.setattr(build, "CSRC", str(csrc))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libgdn.so"))
    monkeypatch.setattr(build, "OBJ", str(tmp_path / "_build"))
    old = 1_000_000_000
    for f in list(csrc.iterdir()) + [tmp_path / "include" / "gdn.h"]:
        os.utime(f, (old, old))
    return tmp_path


def _made(tree):
    """What the compiler was asked to make since the last look."""
    log = tree / "log"
    lines = log.read_text().splitlines() if log.exists() else []
    if log.exists():
        log.unlink()
    return sorted("a" if "a.cu" in x else "b" if "b.cu" in x else "lib" for x in lines)


def _touch(path):
    path.write_text(path.read_text() + "\n")
    os.utime(path, (4_000_000_000, 4_000_000_000))


def test_what_a_change_makes_again(tree, monkeypatch):
    build.build()
    assert _made(tree) == ["a", "b", "lib"]
    build.build()
    assert _made(tree) == []
    monkeypatch.setattr(build, "NVCC_FLAGS", build.NVCC_FLAGS + ["-lineinfo2"])
    build.build()
    assert _made(tree) == ["a", "b", "lib"]            # other flags
    (tree / "version").write_text("two\n")
    build.build()
    assert _made(tree) == ["a", "b", "lib"]            # another compiler
    os.remove(build.LIB)
    build.build()
    assert _made(tree) == ["lib"]
    _touch(tree / "csrc" / "shared.cuh")
    build.build()
    assert _made(tree) == ["a", "lib"]                 # (only the source that includes it)


def test_a_library_without_a_compiler_is_used_as_it_is(tree, monkeypatch):
    build.build()
    monkeypatch.setattr(build, "_nvcc", lambda: str(tree / "no_such_compiler"))
    assert build.up_to_date()


def test_a_failed_build_leaves_nothing_half_made(tree):
    (tree / "fail").write_text("")
    with pytest.raises(subprocess.CalledProcessError):
        build.build()
    time.sleep(1.0)                                    # (a compiler left running would write now)
    assert os.listdir(build.OBJ) == [] and not os.path.exists(build.LIB)
    (tree / "fail").unlink()
    _made(tree)
    build.build()
    assert _made(tree) == ["a", "b", "lib"]
