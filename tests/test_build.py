"""The build on the host, with the compilers replaced: what depends on what."""
import types

import pytest

from chunked_linear_scan_amd import build


def test_the_library_is_linked_where_the_binding_does_not_compile(monkeypatch, tmp_path):
    """The C library needs neither torch's headers nor g++; that the binding failed is still raised."""
    def run(cmd, **_):
        open(cmd[cmd.index("-o") + 1], "w").write("linked")
        return types.SimpleNamespace(returncode=0)

    def no_headers(obj):
        raise RuntimeError("no torch headers")

    lib = tmp_path / "lib.so"
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "HIPCC", __file__)
    monkeypatch.setattr(build, "_compile", lambda src: src + ".o")
    monkeypatch.setattr(build, "_compile_binding", no_headers)
    monkeypatch.setattr(build, "subprocess", types.SimpleNamespace(run=run))
    with pytest.raises(RuntimeError, match="no torch headers"):
        build.build(verbose=False)
    assert lib.read_text() == "linked"
