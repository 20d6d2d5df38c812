"""The build's files while it runs and after it failed, with stand-ins for the
compilers: what is loaded is always a whole library, and nothing is left over."""
import os
import stat

import pytest

TOOL = """#!/bin/sh
# a compiler: notes what stands at the library's place, then writes its output
if [ -e "{lib}" ]; then cat "{lib}" >> "{log}"; else echo absent >> "{log}"; fi
out=
for a in "$@"; do
  case "$last" in -o) out="$a";; esac
  last="$a"
  case "$a" in *{bad}*) exit 1;; esac
done
echo "whole" > "$out"
"""


@pytest.fixture
def b(tmp_path, monkeypatch):
    from gguf_block_quantized_qmatmul_gb300 import build
    folder = tmp_path / "_build"
    monkeypatch.setattr(build, "BUILD", str(folder))
    monkeypatch.setattr(build, "LIB", str(folder / "libqmm.so"))
    monkeypatch.setattr(build, "BINDING", str(folder / "_qmm_torch.so"))
    monkeypatch.setattr(build, "UNITS", ["qmm_api", "qmm_quant"])

    def tools(bad="no such argument"):
        path = tmp_path / "tool"
        path.write_text(TOOL.format(lib=build.LIB, log=tmp_path / "log", bad=f'"{bad}"'))
        path.chmod(path.stat().st_mode | stat.S_IXUSR)
        monkeypatch.setenv("NVCC", str(path))
        monkeypatch.setenv("CXX", str(path))
    build.tools, build.log = tools, tmp_path / "log"
    yield build
    del build.tools, build.log


def left(build):
    return sorted(f for f in os.listdir(build.BUILD) if not f.endswith(".txt"))


def test_no_unfinished_library_is_seen(b):
    b.tools()
    b.build()
    assert set(b.log.read_text().split()) == {"absent"}  # until the last tool was done
    assert left(b) == ["_qmm_torch.so", "libqmm.so"] and b.up_to_date()
    open(b.LIB, "w").write("last build's\n")
    b.build(force=True)
    assert set(b.log.read_text().splitlines()) == {"absent", "last build's"}
    assert open(b.LIB).read() == "whole\n" and left(b) == ["_qmm_torch.so", "libqmm.so"]


@pytest.mark.parametrize("bad", ["qmm_quant.cu", "qmm_torch.cpp", "qmm_api.o"])
def test_a_failed_build_leaves_what_there_was(b, bad):
    b.tools(bad)
    for before in (None, "last build's\n"):
        if before:
            for f in (b.LIB, b.BINDING):
                open(f, "w").write(before)
        with pytest.raises(Exception):
            b.build(force=True)
        assert left(b) == (["_qmm_torch.so", "libqmm.so"] if before else [])
        if before:
            assert open(b.LIB).read() == open(b.BINDING).read() == before
