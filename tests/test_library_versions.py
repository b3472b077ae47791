"""What the binding says of a library of another version (CPU only: stand-ins
built with the host compiler in place of the library)."""
import shutil
import subprocess

import pytest

import moe_layer_align_amd as moe
from test_abi_host import declared_functions

NEW = ("moe_dispatch", "moe_combine", "moe_route_topk_grad", "moe_quant_int8", "moe_swiglu_int8",
       "moe_grouped_gemm_int8", "moe_grouped_int8_workspace_size")


def stand_in(path, version, without=()):
    """A library with the header's functions, which do nothing."""
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    lines = ["int moe_abi_version(void) { return %d; }" % version] if version is not None else []
    lines += ["int %s(void) { return 0; }" % n for n in declared_functions()
              if n != "moe_abi_version" and not n.startswith(tuple(without))]
    src = path.parent / (path.name + ".c")
    src.write_text("\n".join(lines) + "\n")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(path), str(src)], check=True)
    return str(path)


@pytest.mark.parametrize("said,version,without", [
    ("version 14, this binding expects 15: rebuild", 14, ("moe_",)),
    ("version 16, this binding expects 15: rebuild", 16, ()),
    ("moe_dispatch_workspace_size.*rebuild", 15, NEW),
    ("moe_abi_version.*rebuild", None, ()),
])
def test_load_names_a_library_of_another_version(monkeypatch, tmp_path, said, version, without):
    monkeypatch.setattr(moe, "LIB_PATH", stand_in(tmp_path / "libother.so", version, without))
    monkeypatch.setattr(moe, "_lib", None)
    with pytest.raises(RuntimeError, match=said):
        moe.load()
    assert moe._lib is None
