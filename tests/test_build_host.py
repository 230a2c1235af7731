"""The library's build leaves nothing behind but the library."""
import os
import stat

import pytest

from persistent_megakernel_sm_gb300 import build

FAKE = """#!/bin/sh
# a compiler that writes what -o names, and fails where it is told to
out=; last=; link=
while [ $# -gt 0 ]; do
  case "$1" in -o) out="$2"; shift;; -shared) link=1;; esac
  last="$1"; shift
done
echo built > "$out"
case "$link$last" in *{fails}) exit 1;; esac
"""


@pytest.fixture
def compiler(tmp_path, monkeypatch):
    def make(fails):
        path = tmp_path / "nvcc"
        path.write_text(FAKE.replace("{fails}", fails))
        path.chmod(path.stat().st_mode | stat.S_IXUSR)
        monkeypatch.setenv("NVCC", str(path))
        monkeypatch.setattr(build, "LIB", str(tmp_path / "out" / "libmoe.so"))
        return tmp_path / "out"
    return make


def test_a_build_leaves_the_library_alone(compiler):
    out = compiler("nothing")
    assert build.build(force=True) == str(out / "libmoe.so")
    assert os.listdir(out) == ["libmoe.so"]


@pytest.mark.parametrize("fails", ["router.cu", "w4.cu.o"], ids=["a source", "the link"])
def test_a_build_that_fails_leaves_nothing(compiler, fails):
    out = compiler(fails)
    with pytest.raises(Exception):
        build.build(force=True)
    assert os.listdir(out) == []
