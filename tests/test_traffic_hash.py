"""The hash that ties the recorded traffic to the head's code covers every file
that the head's translation unit includes, and changes with each of them."""
import os
import re

import pytest

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = "linear_cross_entropy_tile_amd/csrc/"


def _included():
    """Files of this repository that flce_api.hip includes, itself among them."""
    seen, todo = set(), [CSRC + "flce_api.hip"]
    while todo:
        f = todo.pop()
        if f in seen:
            continue
        seen.add(f)
        with open(os.path.join(ROOT, f), encoding="utf-8") as fh:
            for name in re.findall(r'^#include "([^"]+)"', fh.read(), re.M):
                todo.append("include/flce.h" if name == "flce.h" else CSRC + name)
    return seen


def test_every_included_source_is_hashed():
    assert set(bench.HEAD_SOURCES) == _included()


@pytest.mark.parametrize("source", sorted(_included()))
def test_hash_changes_with_the_code_not_with_comments(source, monkeypatch):
    before, real = bench.kernel_source_hash(), bench._code_only
    with open(os.path.join(ROOT, source), encoding="utf-8") as fh:
        text = fh.read()

    def edited(extra):
        monkeypatch.setattr(bench, "_code_only",
                            lambda t: real(t + extra if t == text else t))
        return bench.kernel_source_hash()

    assert edited("\nint added;\n") != before
    assert edited("\n/* a comment */ // another\n") == before
