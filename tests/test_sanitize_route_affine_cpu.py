"""Host code of routing, combining and the 4-bit products under
AddressSanitizer and UndefinedBehaviorSanitizer (csrc/api_route.cpp and
csrc/api_affine.cpp with the rules that they launch by, compiled with g++ without
device code, driven by tests/sanitize/route_affine_fuzz.cpp): malformed calls are
refused before a launch, accepted ones fit a launch and the workspace that the
library reported for as many rows or more."""
import os
import shutil
import subprocess

import pytest

from tests.test_sanitize_cpu import CSRC, HIP_INC, ROOT


@pytest.fixture(scope="module")
def fuzz_binary(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.isdir(HIP_INC):
        pytest.skip("needs g++ and the HIP headers")
    out = str(tmp_path_factory.mktemp("san") / "route_affine_fuzz")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I", HIP_INC,
           os.path.join(CSRC, "api_route.cpp"), os.path.join(CSRC, "api_affine.cpp"),
           os.path.join(ROOT, "tests", "sanitize", "route_affine_fuzz.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    return out


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_calls_under_sanitizers(fuzz_binary, seed):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([fuzz_binary, "40000", str(seed)], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "runtime error" not in r.stderr and "Sanitizer" not in r.stderr, r.stderr[-4000:]
    words = r.stdout.replace(",", "").split()
    counts = dict((w, int(n)) for n, w in zip(words[2::2], words[3::2]))
    assert counts["accepted"] > 10000 and counts["refused"] > 10000 and counts["launches"] > 10000, r.stdout
