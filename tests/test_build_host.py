"""What building the library needs, and when it builds again (no device)."""
import os

import pytest

from block_scaled_precision_quant_b200 import build


@pytest.fixture
def calls_at(tmp_path, monkeypatch):
    """The compiled calls' place moved to a folder of the test's own."""
    build.build()
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_torch_calls.so"))
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
