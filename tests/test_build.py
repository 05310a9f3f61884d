"""The build's parts (no GPU needed): the library does not wait for the Python module beside it."""
import os

import pytest

from w4a4_quantized_gemm_rudder_amd import build as b


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """Output folders of the test's own, compilers that only leave their output's name."""
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(b, "LIB_DIR", str(tmp_path))
    monkeypatch.setattr(b, "LIB_PATH", str(tmp_path / "librudder.so"))
    monkeypatch.setattr(b, "BIND_PATH", str(tmp_path / "rudder_bind.so"))
    monkeypatch.setattr(b, "generate_tables", lambda: None)
    monkeypatch.setattr(b, "_compile", lambda src: src + ".o")

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done()

    monkeypatch.setattr(b.subprocess, "run", run)
    return tmp_path


def test_library_without_the_module(sandbox, monkeypatch, capsys):
    """Where the module cannot be built (no headers of Python's or torch's, say) the library is,
    with a warning; a module of an earlier build, which may not fit it, is taken away."""
    (sandbox / "rudder_bind.so").touch()

    def fail():
        raise RuntimeError("Python.h: no such file")

    monkeypatch.setattr(b, "build_bind", fail)
    with pytest.warns(UserWarning, match="Python.h"):
        assert b.build() == str(sandbox / "librudder.so")
    assert os.path.exists(sandbox / "librudder.so")
    assert not os.path.exists(sandbox / "rudder_bind.so")
    with pytest.raises(RuntimeError, match="Python.h"):
        b.build(require_bind=True)


def test_library_with_the_module(sandbox, monkeypatch, recwarn):
    b.build()
    assert sorted(os.listdir(sandbox)) == ["librudder.so", "rudder_bind.so"]
    assert not recwarn.list


def test_missing_module_is_an_error(monkeypatch, tmp_path):
    """The operators that need the module raise without it; the linears' calls do not."""
    from w4a4_quantized_gemm_rudder_amd import rudder as r
    r.load_library()
    monkeypatch.setattr(r, "BIND_PATH", str(tmp_path / "rudder_bind.so"))
    monkeypatch.setattr(r, "_bind", None)
    with pytest.raises(r.RudderError, match="rudder_bind.so not found"):
        r.rudder_matvec_w4(1, None, 1, 1, None, None, 0, 64, 128, 64, 1, 1, stream=0)
    assert r.packed_weight_bytes(2048, 6144) > 0
