"""Where the processing of logits counts a token, built with g++ under AddressSanitizer
and UndefinedBehaviorSanitizer (tests/host/process_places_check.cpp)."""
import os
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_tokens_are_counted_inside_the_lds():
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "process_places_check")
        cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
               "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
               "-I" + os.path.join(ROOT, "include"),
               "-I" + os.path.join(ROOT, "linear_cross_entropy_tile_amd", "csrc"),
               os.path.join(ROOT, "tests", "host", "process_places_check.cpp"), "-o", exe]
        subprocess.run(cmd, check=True, capture_output=True, text=True)
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
                   UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
        res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
        assert res.returncode == 0, res.stdout + res.stderr
        assert "failures: 0" in res.stdout, res.stdout
