"""The threshold search's arithmetic (csrc/narrow.h), which the kernels and the
host compile alike, checked on the host under UndefinedBehaviorSanitizer (CPU
only)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_speculative_decoding_router_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_narrowing_on_the_host(tmp_path):
    exe = str(tmp_path / "narrow_host")
    cmd = ["g++", "-std=c++17", "-Wall", "-g", "-O1", "-fsanitize=undefined,float-cast-overflow", "-fno-sanitize-recover=all",
           "-I", CSRC, os.path.join(ROOT, "tests", "host", "narrow_main.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "all checks passed" in r.stdout
