"""CPU sanitizer job of dispatch, combine, their gradients, the grouped products and
their activations (no GPU needed): the host side of their translation units, built
as in test_sanitizers.py, driven by tests/sanitize/abi_tokens_driver.c through
the size helpers and the refusals, with every size and stride at its ends."""
import os
import subprocess

import pytest

from test_sanitizers import CSRC, HERE, HIPCC, HOST_SAN, ROOT, _run

UNITS = ["tokens", "grouped_api", "grouped_tile", "grouped_stream", "grouped_int8"]


@pytest.mark.timeout(600)
def test_tokens_host_paths_under_asan_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    procs = []
    for u in UNITS:
        cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xarch_device", "-O0",
               *HOST_SAN, *inc, "-c", os.path.join(CSRC, u + ".hip"), "-o", str(tmp_path / (u + ".o"))]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
    for cmd, p in procs:
        out, err = p.communicate()
        assert p.returncode == 0, "%s\n%s" % (" ".join(cmd), err[-4000:])
    exe = str(tmp_path / "abi_tokens_driver")
    _run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", *HOST_SAN, *inc, "-x", "c",
          os.path.join(HERE, "abi_tokens_driver.c"), "-x", "none", *[str(tmp_path / (u + ".o")) for u in UNITS],
          "-o", exe])
    res = _run([exe], timeout=300)
    assert "abi tokens sanitizer driver ok" in res.stdout
