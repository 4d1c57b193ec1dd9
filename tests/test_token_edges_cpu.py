"""Edges of the token-path calls that need no GPU to be seen."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "scan_stream_compaction_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")
def test_the_steps_over_the_most_assignments(tmp_path):
    """The row kernels take a token's `per` assignments in sets of 2, 4 or 8:
    the same steps on the host (tests/sets_walk.cpp), up to the largest `per`
    that the calls accept, under the sanitizer of signed overflow. An int that
    steps up by 8 passes its largest value from 2^31 - 7 assignments on."""
    exe = tmp_path / "sets_walk"
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fsanitize=signed-integer-overflow",
                    "-fno-sanitize-recover=all", "-I", CSRC, os.path.join(HERE, "sets_walk.cpp"), "-o", str(exe)],
                   check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout + res.stderr
