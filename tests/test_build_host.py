"""What building the library needs, and when it builds again (no device)."""
import os

import pytest

import block_scaled_precision_quant_b200 as bq
from block_scaled_precision_quant_b200 import build


@pytest.fixture
def calls_at(tmp_path, monkeypatch):
    """The compiled calls' place moved to a folder of the test's own."""
    build.build()
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_torch_calls.so"))
    monkeypatch.setattr(build, "CALLS_STAMP", str(tmp_path / "_torch_calls.built"), raising=False)
    return tmp_path


@pytest.mark.parametrize("cxx", ["/nowhere/g++", "false"])
def test_the_library_is_built_without_the_compiled_calls(calls_at, monkeypatch, cxx):
    """No C++ compiler (or one that fails, as without torch's headers): libbq.so stands."""
    monkeypatch.setenv("CXX", cxx)
    (calls_at / "_torch_calls.so").write_text("of older sources")
    os.utime(build.CALLS, (0, 0))
    with pytest.warns(UserWarning, match="compiled calls are not built"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS)


def test_the_compiled_calls_are_built_again_for_another_torch(calls_at, monkeypatch):
    """They go by the C++ interfaces of one interpreter and one torch."""
    built = []

    def compiler(cmd, **kw):
        built.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("a module")
        return type("Done", (), dict(returncode=0, stdout="", stderr=""))
    monkeypatch.setattr(build.subprocess, "run", compiler)
    for _ in range(2):
        assert build.build_calls() == build.CALLS
    assert len(built) == 1
    version = build.importlib.metadata.version
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: version(name) + ".1")
    for _ in range(2):
        build.build_calls()
    assert len(built) == 2
    var = build.sysconfig.get_config_var
    monkeypatch.setattr(build.sysconfig, "get_config_var",
                        lambda name: "cpython-999" if name == "SOABI" else var(name))
    for _ in range(2):
        build.build_calls()
    assert len(built) == 3


def test_compiled_calls_of_another_torch_are_not_loaded(calls_at, monkeypatch):
    (calls_at / "_torch_calls.so").write_text("a module")
    (calls_at / "_torch_calls.built").write_text("cpython-999 torch 0.1")
    monkeypatch.setattr(bq, "_native", None)
    with pytest.raises(RuntimeError, match="not built for"):
        bq.act_quant_int8(None)
