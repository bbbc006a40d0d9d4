"""Which of the 4-bit layer's forms the GPU tests' shapes take (csrc/narrow/fp4_forms.h, compiled
here), so that none of them is left without a test when the rule changes."""
import os
import subprocess

import pytest

from test_gpu_fp4 import LAYERS
from test_gpu_fp4_forms import FORMS, LINES, ONES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NARROW = os.path.join(ROOT, "dlrm_embedding_bag_b200", "csrc", "narrow")
SMS = 148  # of a B200

ASK = r"""
#include <cstdio>
#include "fp4_forms.h"
int main() {
  long long m, k, n;
  int lines;
  while (std::scanf("%lld %lld %lld %d", &m, &k, &n, &lines) == 4) {
    const long long even = (k + 1) / 2 * 2;  // as the binding has it: whole bytes
    if (dlrm::fp4_one_token(m, n, even)) {
      const dlrm::Fp4One v = dlrm::kFp4OneOf[dlrm::fp4_one(n, static_cast<int>((even + 31) / 32), SMS)];
      std::printf("one %d %d 0\n", v.blocks, v.channels);
    } else {
      const dlrm::Fp4Form f = dlrm::kFp4FormOf[dlrm::fp4_form(m, n, static_cast<int>((even + 255) / 256), lines != 0, SMS)];
      std::printf("tiles %d %d %d\n", f.rows_n, f.split, f.lines ? 1 : 0);
    }
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    """shapes, whether rows of y are whole 16 bytes -> [(kind, a, b, lines)]."""
    at = tmp_path_factory.mktemp("forms")
    (at / "ask.cpp").write_text(ASK)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", f"-DSMS={SMS}", "-I", NARROW,
                    str(at / "ask.cpp"), "-o", str(at / "ask")], check=True)

    def call(shapes, lines):
        said = subprocess.run([str(at / "ask")], input="".join(f"{m} {k} {n} {int(lines)}\n" for m, k, n in shapes),
                              capture_output=True, text=True, check=True).stdout.split("\n")[:-1]
        assert len(said) == len(shapes)
        return [(kind, int(a), int(b), int(c)) for kind, a, b, c in (line.split() for line in said)]

    return call


def test_shapes_take_the_forms_that_they_stand_for(ask):
    for kind, table in (("tiles", FORMS), ("one", ONES)):
        for form, shapes in table.items():
            assert ask(shapes, False) == [(kind, *form, 0)] * len(shapes), form


def test_outputs_that_leave_as_whole_lines(ask):
    assert ask(LINES, True) == [("tiles", 256, 1, 1)] * len(LINES)


def test_no_form_is_without_a_test(ask):
    """All kernels that the dispatch can take, whole lines by the outputs that are whole lines."""
    source = open(os.path.join(NARROW, "fp4_forms.h")).read()
    assert "kFp4Forms = 8;" in source and "kFp4Ones = 5;" in source
    tested = {("tiles", *f, 0) for f in FORMS} | {("one", *f, 0) for f in ONES}
    assert len(tested) == 8 - 1 + 5
    whole = [s for s in LAYERS if s[2] % 8 == 0]
    assert set(ask(whole, True)) - tested == {("tiles", 256, 1, 1)}
    assert set(ask(LAYERS, False)) <= tested
