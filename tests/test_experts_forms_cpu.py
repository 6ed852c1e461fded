"""Which kernel forms the GPU tests of the grouped products run: the rules of
csrc/expert_choice.hpp, compiled with g++, name the form of every size that
tests/test_gpu_experts.py multiplies, and every form of every type and layout has
to be among them.  A change of the rules that leaves a form without a size
fails here (no GPU)."""
import os
import re
import shutil
import subprocess

import pytest

from tests import test_gpu_experts as gx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "adapter_lora_segments_amd", "csrc")
HIP_INC = "/opt/rocm/include"

TABLES = {"bf16 nk": ("kBf16Nk", 2.0), "bf16 kn": ("kBf16Kn", 2.0), "fp32 nk": ("kF32Nk", 4.0),
          "fp32 kn": ("kF32Kn", 4.0), "w4 bf16": ("kW4A16", 17 / 32), "w4 mxfp4": ("kW4A4", 17 / 32)}

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include "expert_choice.hpp"
using namespace mlora;
template <int N>
void say(const Choice (&t)[N], bool fixed, double per, const ExpertArgs& a) {
  const Choice& c = choose(t, fixed, a, per * a.K * a.N);
  std::printf("%s%dx%d\n", c.few ? "few " : "", c.rows, c.cols);
}
template <int N>
void all(const char* name, const Choice (&t)[N]) {
  for (const Choice& c : t) std::printf("%s %s%dx%d\n", name, c.few ? "few " : "", c.rows, c.cols);
}
int main(int argc, char** argv) {
  if (argc == 1) {
    all("kBf16Nk", kBf16Nk), all("kBf16Kn", kBf16Kn), all("kF32Nk", kF32Nk), all("kF32Kn", kF32Kn);
    all("kW4A16", kW4A16), all("kW4A4", kW4A4);
  }
  for (int i = 1; i + 5 < argc; i += 6) {       // table, bytes a weight, rows, experts, K, N
    const int32_t one = 0;
    ExpertArgs a{};
    a.rows = std::atoi(argv[i + 2]), a.n_experts = std::atoi(argv[i + 3]);
    a.K = std::atoi(argv[i + 4]), a.N = std::atoi(argv[i + 5]);
    a.offsets = &one;
    const double per = std::atof(argv[i + 1]);
    if (!std::strcmp(argv[i], "dW")) std::printf("%d\n", dw_tile(per > 2, a.rows, a.K, a.N));   // rows: the experts
    else if (!std::strcmp(argv[i], "kBf16Nk")) say(kBf16Nk, false, per, a);
    else if (!std::strcmp(argv[i], "kBf16Kn")) say(kBf16Kn, false, per, a);
    else if (!std::strcmp(argv[i], "kF32Nk")) say(kF32Nk, true, per, a);
    else if (!std::strcmp(argv[i], "kF32Kn")) say(kF32Kn, true, per, a);
    else if (!std::strcmp(argv[i], "kW4A16")) say(kW4A16, false, per, a);
    else say(kW4A4, false, per, a);
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
        args = [str(v) for q in queries for v in q]
        return subprocess.run([str(d / "forms")] + args, capture_output=True, text=True, check=True).stdout.splitlines()
    return ask


def taken(rules, kind, sizes):
    name, per = TABLES[kind]
    return rules([(name, per, r, e, di, do) for r, e, di, do in sizes])


@pytest.mark.parametrize("kind", list(TABLES))
def test_every_form_has_a_size(rules, kind):
    """Over short reductions and long ones, whole and (bf16, fp32) ending inside
    a step; MXFP4 x MXFP4 for both alignments of the scales."""
    every = {l.split(" ", 1)[1] for l in rules([]) if l.startswith(TABLES[kind][0] + " ")}
    sizes = gx.FORMS[kind]
    got = taken(rules, kind, sizes)
    assert set(got) == every
    if kind[0] != "w":
        odd = [s for f, s in gx.ODD if f == kind]
        step = 64 if kind.startswith("bf16") else 32
        assert all(di % step for _, _, di, _ in odd)
        assert set(taken(rules, kind, odd)) == every
    if kind == "w4 mxfp4":
        pairs = {(f, di % 512 == 0) for f, (_, _, di, _) in zip(got, sizes)}
        few = {f for f in every if f.startswith("few")}
        assert {f for f, whole in pairs if whole} | few == every        # (few-row forms know one alignment)
        assert {f for f, whole in pairs if not whole} == every


def test_every_table_entry_has_a_kernel():
    """The dispatch names each tile of the tables; what it does not name falls
    through to its last line's tile."""
    src = open(os.path.join(CSRC, "kernels_expert.hip")).read()
    tables = open(os.path.join(CSRC, "expert_choice.hpp")).read()
    tiles = {(int(r), int(c)) for r, c in re.findall(r"\{false, (\d+), (\d+),", tables)}
    named = {(64 * int(f), 64 * int(n)) for f, n in re.findall(r"rows_(?:pipe<AL, BL|f32_tile<BL), (\d), (\d)>\(a, s\)", src)}
    assert tiles == named


def test_every_gradient_tile_has_a_size(rules):
    """dW: the sizes of test_backward, test_gradients_of_wide_weights."""
    narrow = [(dt, len(s), di, do) for dt, pad in (("bf16", 0), ("fp32", 4)) for s in gx.SIZES.values()
              for di, do in ((a + pad, b + pad) for a, b in gx.DIMS)]
    mark = next(m for m in gx.test_gradients_of_wide_weights.pytestmark if m.name == "parametrize" and "dt" in m.args[0])
    wide = [(dt, len(s), di, do) for dt, di, do, s in mark.args[1]]
    got = {}
    for dt, e, di, do in narrow + wide:
        per = 4.0 if dt == "fp32" else 2.0
        got.setdefault(dt, set()).update(int(v) for v in rules([("dW", per, e, 1, di, do), ("dW", per, e, 1, do, di)]))
    assert got == {"bf16": {128, 256}, "fp32": {64, 128, 256}}
