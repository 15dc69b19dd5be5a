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
