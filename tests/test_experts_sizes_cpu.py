"""Sizes that the grouped products compute in 32 bits, at the largest shapes the
C interface takes (host functions of csrc/experts.hpp, compiled with g++ and
checked against 64-bit arithmetic; no GPU)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from adapter_lora_segments_amd import _lib
from tests.test_experts_cpu import shape

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "adapter_lora_segments_amd", "csrc")
HIP_INC = "/opt/rocm/include"

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include "experts.hpp"
// (an overflow in a constant expression does not compile)
static_assert(mlora::pieces_of(2147483391, 8388608) == 256, "");
static_assert(mlora::pieces_of(2147483647, 2147483647) == 1, "");
static_assert(mlora::pieces_of(0, 256) == 0 && mlora::pieces_of(1, 256) == 1 && mlora::pieces_of(256, 256) == 1 &&
              mlora::pieces_of(257, 256) == 2, "");
int main(int argc, char** argv) {
  // f32 rows experts m n -> chunk, pieces of one group of all rows, pieces of
  // two halves, bytes of the partial sums
  for (int i = 1; i + 4 < argc; i += 5) {
    const bool f32 = std::atoi(argv[i]);
    const long long rows = std::atoll(argv[i + 1]), e = std::atoll(argv[i + 2]), m = std::atoll(argv[i + 3]),
                    n = std::atoll(argv[i + 4]);
    const long long c = mlora::dw_chunk(f32, rows, e, m, n);
    const int half = (int)(rows / 2);
    std::printf("%lld %d %d %d %lld\n", c, c ? mlora::pieces_of((int)rows, (int)c) : 0,
                c ? mlora::pieces_of(half, (int)c) : 0, c ? mlora::pieces_of((int)rows - half, (int)c) : 0,
                (long long)mlora::dw_part_bytes(f32, rows, e, m, n));
  }
}
"""


def most_rows(**kw):
    """The largest number of rows that the interface accepts."""
    L, n = _lib.lib(), ctypes.c_int64()
    lo, hi = 0, 1 << 31
    while lo + 1 < hi:
        mid = (lo + hi) // 2
        if L.mlora_expert_workspace(ctypes.byref(shape(rows=mid, **kw)), ctypes.byref(n)) == 0:
            lo = mid
        else:
            hi = mid
    return lo


def test_chunk_counts_at_the_largest_rows(tmp_path):
    if shutil.which("g++") is None or not os.path.isdir(HIP_INC):
        pytest.skip("needs g++ and the HIP headers")
    src, exe = tmp_path / "sizes.cpp", tmp_path / "sizes"
    src.write_text(DRIVER)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I", HIP_INC, "-I", CSRC,
                        str(src), "-o", str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    cases = []
    for dtype in (0, 1):
        for E in (1, 2, 100):
            for d in ((8, 8), (128, 128), (8, 264), (264, 520)):
                top = most_rows(dtype=dtype, n_experts=E, d_in=d[0], d_out=d[1])
                # the largest launch: rows / 256 + E tiles of rows, times those along N
                assert top == ((1 << 23) - 1) // ((max(d) + 255) // 256) * 256 - 256 * E + 255, (top, d, E)
                cases += [(1 - dtype, rows, E, *d) for rows in (top, top - 1, top // 2, top // 256 * 255, 10 ** 6)]
    out = subprocess.run([str(exe)] + [str(v) for c in cases for v in c], capture_output=True, text=True, check=True)
    lines = out.stdout.splitlines()
    assert len(lines) == len(cases)
    for (f32, rows, E, m, n), line in zip(cases, lines):
        c, all_rows, a, b, room = map(int, line.split())
        t = -(-m // 128) * -(-n // 128)
        want = max(-(-(-(-rows * t // 256)) // 64) * 64, 256 if f32 else 1024)
        assert c == (0 if E * t >= 256 or rows <= want else want), (f32, rows, E, m, n, c)
        if c:
            assert all_rows == -(-rows // c) and a == -(-(rows // 2) // c) and b == -(-(rows - rows // 2) // c)
            # a slot for every chunk of every group that has several
            for slots in (all_rows, (a if a > 1 else 0) + (b if b > 1 else 0)):
                assert slots <= 2 * rows // c and slots * m * n * 4 <= room
