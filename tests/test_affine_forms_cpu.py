"""Which kernel forms the GPU tests of the 4-bit products run: the rules of
csrc/affine_choice.hpp, compiled with g++, name the form of every size that
tests/test_gpu_affine_forms.py multiplies for that purpose, and every form has to be
among them; and every form that the rules name has a kernel (no GPU)."""
import os
import re
import shutil
import subprocess

import pytest

from tests import test_gpu_affine_forms as ga

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "adapter_lora_segments_amd", "csrc")
HIP_INC = "/opt/rocm/include"

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include "affine_choice.hpp"
using namespace mlora;
void say(const AffineChoice& c) { std::printf("%s %dx%dx%d\n", c.few ? "few" : "tile", c.rows, c.cols, c.split); }
int main(int argc, char** argv) {
  if (argc == 1) {
    for (const AffineChoice& c : kAffine) say(c);
    std::printf("dx\n");
    for (const AffineChoice& c : kAffineDx) say(c);
  }
  for (int i = 1; i + 5 < argc; i += 6) {       // dx, rows, experts, d_in, d_out, group
    const int32_t one = 0;
    const bool dx = std::atoi(argv[i]) != 0;
    ExpertArgs a{};
    a.rows = std::atoi(argv[i + 1]), a.n_experts = std::atoi(argv[i + 2]);
    a.K = std::atoi(argv[i + 3 + dx]), a.N = std::atoi(argv[i + 4 - dx]);
    a.offsets = &one;
    const int g = std::atoi(argv[i + 5]);
    say(dx ? affine_choose(kAffineDx, a, g) : affine_choose(kAffine, a, g));
  }
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.isdir(HIP_INC):
        pytest.skip("needs g++ and the HIP headers")
    d = tmp_path_factory.mktemp("forms")
    (d / "forms.cpp").write_text(DRIVER)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I", HIP_INC, "-I", CSRC,
                        str(d / "forms.cpp"), "-o", str(d / "forms")], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr

    def ask(queries):
        args = [str(int(v)) for q in queries for v in q]
        return subprocess.run([str(d / "forms")] + args, capture_output=True, text=True, check=True).stdout.splitlines()
    return ask


def test_every_form_has_a_size(rules):
    lines = rules([])
    fwd, dx = lines[:lines.index("dx")], lines[lines.index("dx") + 1:]
    assert set(ga.FORMS) == set(fwd) and set(ga.DX_FORMS) == set(dx)
    for g in (32, 64, 128):
        assert rules([(0,) + v + (g,) for v in ga.FORMS.values()]) == list(ga.FORMS)
        assert rules([(1,) + v + (g,) for v in ga.DX_FORMS.values()]) == list(ga.DX_FORMS)


def test_few_rows_are_never_rounded(rules):
    """Up to 16 rows a group the few-row kernel, whatever the sizes."""
    q = [(0, r * e, e, di, do, 128) for r in (1, 4, 16) for e in (1, 8, 300) for di in (128, 4096, 1 << 18)
         for do in (8, 14336, 1 << 18)]
    assert all(f.startswith("few") for f in rules(q))


def test_every_entry_has_a_kernel(rules):
    """The dispatch names each tile of the lists; what it does not name falls through to its last line's."""
    src = open(os.path.join(CSRC, "kernels_affine.hip")).read()
    few = {(int(r), 16 * int(n) * int(c)) for r, n, c in re.findall(r"few_of<(\d+), (\d+), (\d+)>\(a", src)}
    src = open(os.path.join(CSRC, "kernels_affine_tile.hip")).read()
    tile = {(32 * int(f), int(k)) for f, k in re.findall(r"tile_of<(\d+), (\d+)>\(a", src)}
    dx = {(32 * int(f), int(k)) for f, k in re.findall(r"dx_of<(\d+), (\d+)>\(a", src)}
    want = {"few": set(), "tile": set(), "dx": set()}
    kind = None
    for l in rules([]):
        if l == "dx":
            kind = "dx"
            continue
        k, (r, c, s) = l.split()[0], (int(v) for v in l.split()[1].split("x"))
        want[kind or k].add((r, c) if k == "few" else (r, s))
    assert want == {"few": few, "tile": tile, "dx": dx}
