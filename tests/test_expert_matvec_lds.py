"""The LDS layout of the expert products' kernel, checked on the host over every form, wave, step and lane."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_stores_and_reads_lie_in_the_x(tmp_path):
    exe = str(tmp_path / "lds")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "moe_routing_fp8_amd", "csrc"),
                    os.path.join(ROOT, "tests", "layout", "expert_matvec_lds.cpp"), "-o", exe], check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout
