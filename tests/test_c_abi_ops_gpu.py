"""The operators beside the head from plain C99: tests/c_abi/flce_ops_check.c,
built like the head's program with gcc against include/flce.h and the in-tree
library, checks them against their definitions. Run here as a child process."""
import os
import subprocess

import pytest

pytestmark = pytest.mark.gpu

BIN = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c_abi", "flce_ops_check")


def test_c_program():
    assert os.path.exists(BIN), f"{BIN} missing: run __graft_entry__.build() first"
    res = subprocess.run([BIN], capture_output=True, text=True, timeout=120)
    print(res.stdout, res.stderr, flush=True)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "flce_ops_check ok" in res.stdout
