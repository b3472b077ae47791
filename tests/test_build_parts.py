"""The C ABI's libraries do not depend on what the binding's compiled part needs
(CPU only: stand-ins in place of the compiles)."""
import sys

import pytest

from moe_layer_align_amd import build


@pytest.fixture
def linked(monkeypatch):
    """Names of the libraries in the order in which they are linked."""
    done = []

    def compile_link(units, lib, *_):
        return lambda: done.append(lib)
    monkeypatch.setattr(build, "_compile_link", compile_link)
    return done


def test_libraries_without_a_host_compiler(monkeypatch, linked):
    monkeypatch.setattr(build, "CXX", "/nonexistent/c++")
    with pytest.raises(RuntimeError, match="binding's compiled part.*libraries are built"):
        build.build()
    assert linked == [build.LIB, build.PROBE_LIB]


@pytest.mark.parametrize("name", ["torch", "torch.utils.cpp_extension"])
def test_libraries_without_torch(monkeypatch, linked, name):
    monkeypatch.setitem(sys.modules, name, None)  # makes its import fail
    with pytest.raises(RuntimeError, match="binding's compiled part.*libraries are built"):
        build.build()
    assert linked == [build.LIB, build.PROBE_LIB]


def test_a_failing_library_is_the_error(monkeypatch, linked):
    def compile_link(units, lib, *_):
        def finish():
            raise RuntimeError("hipcc failed on %s" % units[0])
        return finish
    monkeypatch.setattr(build, "_compile_link", compile_link)
    monkeypatch.setattr(build, "CXX", "/nonexistent/c++")
    with pytest.raises(RuntimeError, match="hipcc failed"):
        build.build()
