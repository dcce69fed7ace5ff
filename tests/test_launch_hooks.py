"""The launch hooks under an allocator that fails (tests/host/launch_check.cpp),
built with g++ against the HIP headers with stand-ins for the event calls."""
import os
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("g++") is None
                    or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")),
                    reason="g++ or the HIP headers not available")
def test_no_exception_leaves_the_launch_hooks():
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "launch_check")
        cmd = ["g++", "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__",
               "-I" + os.path.join(ROCM, "include"), "-I" + os.path.join(ROOT, "include"),
               "-I" + os.path.join(ROOT, "linear_cross_entropy_tile_amd", "csrc"),
               os.path.join(ROOT, "tests", "host", "launch_check.cpp"), "-o", exe]
        res = subprocess.run(cmd, capture_output=True, text=True)
        assert res.returncode == 0, res.stderr
        res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
        assert res.returncode == 0 and "failures: 0" in res.stdout, res.stdout + res.stderr
