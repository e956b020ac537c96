"""What build() compiles, with the compiler replaced: the library, the binding, or neither."""
import importlib.util
import os

import pytest

from weight_quantized_gemm_anti_b200 import buildlib


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """Names of what the compiler was asked for, in a package folder of its own with an up-to-date build."""
    asked = []

    def run(cmd, check=True, **kw):
        out = cmd[cmd.index("-o") + 1]
        asked.append(os.path.basename(out).replace(".tmp", ""))
        open(out, "w").close()

    src = tmp_path / "csrc"
    src.mkdir()
    for name in ("api.cu", "binding.cpp", "host.h"):
        (src / name).write_text("")
        os.utime(src / name, (1, 1))
    monkeypatch.setattr(buildlib, "HERE", str(tmp_path))
    monkeypatch.setattr(buildlib, "CSRC", str(src))
    monkeypatch.setattr(buildlib, "LIB", str(tmp_path / "libwqmm.so"))
    monkeypatch.setattr(buildlib, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(buildlib, "SOURCES", ["api.cu"])
    monkeypatch.setattr(buildlib.subprocess, "run", run)
    buildlib.build()
    assert sorted(asked) == ["_binding.so", "api.o", "libwqmm.so"]
    asked.clear()
    return asked


def later(path):
    """The file is newer than all that was built."""
    t = max(os.path.getmtime(f) for f in (buildlib.LIB, buildlib.BINDING)) + 10
    os.utime(path, (t, t))


def test_up_to_date(compiled):
    assert buildlib.build() == buildlib.LIB
    assert compiled == []


def test_a_binding_that_is_missing_is_all_that_is_built(compiled):
    os.remove(buildlib.BINDING)
    buildlib.build()
    assert compiled == ["_binding.so"]


def test_a_source_of_the_binding_alone(compiled):
    later(os.path.join(buildlib.CSRC, "binding.cpp"))
    buildlib.build()
    assert compiled == ["_binding.so"]


def test_a_source_of_the_library(compiled):
    later(os.path.join(buildlib.CSRC, "host.h"))
    buildlib.build()
    assert "libwqmm.so" in compiled and "api.o" in compiled


@pytest.mark.parametrize("what", ["torch", "python"])
def test_another_torch_or_python(compiled, monkeypatch, what):
    """The binding is built for one interpreter and one torch: under another it is built anew."""
    torch = pytest.importorskip("torch")
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "9.9.9")
    else:
        monkeypatch.setattr(buildlib.sysconfig, "get_config_var", lambda name: "cpython-999")
    buildlib.build()
    assert compiled == ["_binding.so"]
    buildlib.build()
    assert compiled == ["_binding.so"]


def test_without_torch(compiled, monkeypatch, capsys):
    """The library needs nvcc alone; there is no binding then, and build() says so."""
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setitem(buildlib.sys.modules, "torch", None)
    os.remove(buildlib.BINDING)
    assert buildlib.build() == buildlib.LIB and compiled == []
    os.remove(buildlib.LIB)
    assert buildlib.build() == buildlib.LIB
    assert "libwqmm.so" in compiled and "_binding.so" not in compiled
    assert "torch" in capsys.readouterr().err
