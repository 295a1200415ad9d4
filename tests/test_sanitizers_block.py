"""AddressSanitizer and UndefinedBehaviorSanitizer on the host side of the block operators' entry points (CPU only;
nothing here runs on a GPU): their sources and tests/sanitize/block_driver.cpp."""
import os
import subprocess

import pytest

from test_sanitizers import CLANG, HIPCC, ROOT, SAN, _host_san_flags, _run

SOURCES = ["block_norm.hip", "balance_loss.hip", "expert_matvec.hip", "moe_fp8_api.hip"]


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm toolchain not available")
def test_host_block_operators_under_asan_and_ubsan(tmp_path):
    csrc = os.path.join(ROOT, "moe_routing_fp8_amd", "csrc")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", csrc]
    files = [os.path.join(csrc, name) for name in SOURCES]
    files.append(os.path.join(ROOT, "tests", "sanitize", "block_driver.cpp"))
    objs = [str(tmp_path / (os.path.basename(f) + ".o")) for f in files]
    procs = [subprocess.Popen([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", *_host_san_flags(),
                               "-Xarch_device", "-O1", *inc, "-c", f, "-o", o],
                              stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
             for f, o in zip(files, objs)]
    for p in procs:
        out, _ = p.communicate(timeout=600)
        assert p.returncode == 0, out
    exe = str(tmp_path / "block_san")
    # moe_fp8_api.hip, for the status of a HIP error, names launches of other sources; none is reached
    rc, log = _run([CLANG, *SAN, *objs, "-Wl,--unresolved-symbols=ignore-all", "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    assert rc == 0, log
    rc, log = _run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert rc == 0 and log.strip().endswith("ok"), log
