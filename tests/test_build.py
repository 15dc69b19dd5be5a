"""What build.py makes, and when."""
import os
import sysconfig

import pytest
import torch

from pagedattention_kv_cache_attention_gb300 import build


def test_binding_is_named_for_its_torch_and_its_python():
    name = os.path.basename(build.BIND)
    assert torch.__version__ in name
    assert name.endswith("." + sysconfig.get_config_var("SOABI") + ".so")


@pytest.fixture
def tools(monkeypatch, tmp_path):
    """build.py with a folder of its own and compilers that only write what they would have made;
    the names of what they were asked for."""
    made, run = [], build.subprocess.run

    def compiler(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        made.append(os.path.basename(out).split(".so")[0].split(".o")[0])
        open(out, "w").close()
        return run(["true"], **kw)

    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libpa.so"))
    monkeypatch.setattr(build, "BIND", str(tmp_path / os.path.basename(build.BIND)))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(build.subprocess, "run", compiler)
    return made


def test_library_is_linked_where_the_binding_does_not_compile(tools, monkeypatch):
    def fails(*args):
        raise RuntimeError("Python.h: No such file or directory")
    monkeypatch.setattr(build, "_compile_bind", fails)
    with pytest.raises(RuntimeError, match="libpa.so is built.*Python.h"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BIND)
    assert set(tools) == {s[:-3] for s in build.SOURCES} | {"libpa"}


def test_only_what_is_out_of_date_is_made(tools, monkeypatch, tmp_path):
    lib = {s[:-3] for s in build.SOURCES} | {"libpa"}

    def made():
        tools.clear()
        build.build()
        return set(tools)

    assert made() == lib | {"pa_bind", os.path.basename(build.BIND)[:-3]}
    assert made() == set()
    # another torch or another Python: another file
    monkeypatch.setattr(build, "BIND", str(tmp_path / "pa_bind-other.so"))
    assert made() == {"pa_bind", "pa_bind-other"}
    assert made() == set()
    # sources newer than one of the two
    csrc, include = tmp_path / "csrc", tmp_path / "include"
    csrc.mkdir(), include.mkdir()
    monkeypatch.setattr(build, "CSRC", str(csrc))
    monkeypatch.setattr(build, "HERE", str(tmp_path / "package"))
    for f in (*build.SOURCES, "pa_tile.cuh", "pa_internal.h", "pa_bind.cpp", "../include/pa.h"):
        (csrc / f).touch()
        os.utime(csrc / f, (0, 0))
    now = os.path.getmtime(build.LIB) + 100
    assert made() == set()
    for f, want in (("pa_bind.cpp", {"pa_bind", "pa_bind-other"}), ("pa_tile.cuh", lib),
                    ("pa_sparse.cu", lib), ("../include/pa.h", lib | {"pa_bind", "pa_bind-other"})):
        os.utime(csrc / f, (now, now))
        assert made() == want, f
        os.utime(csrc / f, (0, 0))
