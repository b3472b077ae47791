"""What the binding says of a library of another version (CPU only: stand-ins
built with the host compiler in place of the library)."""
import os
import re
import shutil
import subprocess
import sys

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


CALLS = """
import importlib.util, sys
import torch
spec = importlib.util.spec_from_file_location("_calls", sys.argv[1])
try:
    calls = importlib.util.module_from_spec(spec)
    calls.init(None, None, None, None)
    print("fits")
except (ImportError, RuntimeError) as e:
    print(type(e).__name__, e)
"""


@pytest.mark.parametrize("said,version,without", [
    ("fits", 15, ()),
    ("RuntimeError libmoe_mi355x.so has ABI version 14, the binding's compiled part is of version 15: rebuild", 14, ()),
    ("ImportError.*undefined symbol: moe_", 15, NEW),
])
def test_the_compiled_part_compares_versions(tmp_path, said, version, without):
    # beside another library than its own, in a process that holds neither
    part = os.path.join(os.path.dirname(moe.LIB_PATH), "_calls.so")
    shutil.copy(part, tmp_path / "_calls.so")
    stand_in(tmp_path / os.path.basename(moe.LIB_PATH), version, without)
    res = subprocess.run([sys.executable, "-c", CALLS, str(tmp_path / "_calls.so")], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    assert re.search(said, res.stdout), res.stdout
