"""The line of key tiles that paged attention cuts among its CTAs, its arithmetic compiled for the
host: stretches cover the line, every unit's CTA is found, and sums that pass 31 bits are seen
instead of wrapping (a part's place in the workspace would lie behind it)."""
import os
import shutil
import subprocess

import pytest

from gated_delta_rule_55_gb300 import build_lib

MAIN = r"""
#include <cstdio>
#include "kda_paged_line.h"
using namespace kda;
int main() {
  char op;
  int a, b;
  while (std::scanf(" %c %d %d", &op, &a, &b) == 3)
    std::printf("%d\n", op == 's' ? stretch(a, b) : op == 'o' ? stretch_of(a, b) : line_add(a, b));
}
"""
CTAS, MOST = 152, 2 ** 31 - 1


@pytest.fixture(scope="module")
def line(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("line")
    (d / "main.cpp").write_text(MAIN)
    csrc = os.path.join(build_lib.PKG, "csrc")
    subprocess.run([cxx, "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", csrc,
                    str(d / "main.cpp"), "-o", str(d / "line")], check=True)

    def ask(queries):
        text = "\n".join(f"{o} {a} {b}" for o, a, b in queries)
        r = subprocess.run([str(d / "line")], input=text, capture_output=True, text=True,
                           check=True)
        return [int(x) for x in r.stdout.split()]
    return ask


@pytest.mark.parametrize("total", [0, 1, 3, 151, 152, 153, 303, 304, 305, 100_001, 2 ** 30,
                                   MOST - 1])
def test_stretches_and_their_units(line, total):
    at = line([("s", total, c) for c in range(CTAS + 1)])
    assert at[0] == 0 and at[-1] == total
    assert all(0 <= b - a <= total // CTAS + 1 for a, b in zip(at, at[1:]))
    units = sorted({u for a in at for u in (a - 1, a, a + 1) if 0 <= u < total})
    own = line([("o", total, u) for u in units])
    assert all(at[c] <= u < at[c + 1] for u, c in zip(units, own))


def test_sums_stop_instead_of_wrapping(line):
    pairs = [(0, 0), (1, 2), (MOST - 1, 0), (MOST - 2, 1), (MOST - 1, 1), (2 ** 30, 2 ** 30),
             (MOST, 0), (MOST, MOST), (MOST - 1, MOST - 1)]
    assert line([("+", a, b) for a, b in pairs]) == [min(a + b, MOST) for a, b in pairs]


def test_a_long_line_of_overlapping_sequences_is_seen(line):
    """Every other of 8192 sequences with all 4096 tokens and keys, 3500 heads: 2^32 units and
    more, each sequence's inside 31 bits.  The 32-bit sum is a small positive number."""
    per = 3500 * sum((256 * rt + 255) // 128 + 1 + 2 for rt in range(16))
    assert 2 ** 32 < 4096 * per and 0 < 4096 * per - 2 ** 32 < 2 ** 31 and per < MOST
    total = 0
    for k in range(12):  # doubling: 2^12 sequences
        total = line([("+", total or per, total or per)])[0]
    assert total == MOST
