"""The planning of the operators for prompts (csrc/plan.h) built with g++ under
AddressSanitizer and UndefinedBehaviorSanitizer, and the tile rule against the
tests' copy of it (CPU only)."""
import os
import random
import shutil
import subprocess

import pytest

from plan_rules import tile_rows

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
CSRC = os.path.join(ROOT, "moe_speculative_decoding_router_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(os.path.join(ROCM, "include", "hip")),
                    reason="needs g++ and the HIP headers")
def test_planning_on_the_host(tmp_path):
    exe = str(tmp_path / "plan_host")
    cmd = ["g++", "-std=c++17", "-w", "-g", "-O1", "-D__HIP_PLATFORM_AMD__", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I", os.path.join(ROCM, "include"), "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(ROOT, "tests", "host", "plan_main.cpp"),
           "-L", os.path.join(ROCM, "lib"), "-lamdhip64", f"-Wl,-rpath,{os.path.join(ROCM, 'lib')}", "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    rnd = random.Random(1)
    calls = [(T, k, E, 32 * i, f) for T in (1, 27, 28, 64, 127, 128, 896, 4096) for k in (1, 2) for E in (1, 2, 32, 64, 128) for i in (1, 8, 17, 260)
             for f in (0, 1)]
    calls += [(rnd.randint(1, 1 << 20), rnd.randint(1, 32), rnd.randint(32, 512), 32 * rnd.randint(1, 300), rnd.randint(0, 1)) for _ in range(500)]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], input="\n".join(" ".join(map(str, c)) for c in calls), capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.stdout[-500:] + r.stderr)[-4000:]
    lines = r.stdout.split("\n")
    assert "all checks passed" in lines
    assert [int(x) for x in lines[:len(calls)]] == [tile_rows(*c) for c in calls]
    assert {tile_rows(*c) for c in calls} == {32, 128, 256}
