"""The kernel that each tested size of the fused products takes (no GPU needed): the
choice compiled for the host, so that a change of the modelled times cannot take a
kernel out of the tests unseen."""
import os
import shutil
import subprocess

import pytest

from micro_scaled_fp4_amd import build
from product_sizes import DENSE, GROUPED, SHORT

CUS = 256                                # compute units of an MI355X

MAIN = """
#include <stdio.h>
#include "product_choice.h"
int main() {
  int mx, cus;
  long long g, M, N, K;
  while (scanf("%d %lld %lld %lld %lld %d", &mx, &g, &M, &N, &K, &cus) == 6)
    printf("%d\\n", fp4impl::choose_rows(mx != 0, g, M, N, K, cus));
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("choice")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", f"-I{build.CSRC}", str(d / "main.cpp"), "-o", str(d / "choice")],
                   check=True)

    def run(cases):
        text = "".join(" ".join(map(str, c)) + "\n" for c in cases)
        out = subprocess.run([str(d / "choice")], input=text, capture_output=True, text=True, check=True, timeout=60).stdout
        return [int(x) for x in out.split()]
    return run


def test_every_listed_size_takes_its_kernel(choose):
    cases = [(int(f == "mx"), 0, M, N, K, CUS) for _, f, M, N, K in DENSE + SHORT]
    cases += [(int(f == "mx"), len(s), sum(s) + tail, N, K, CUS) for _, f, s, tail, N, K in GROUPED]
    got = choose(cases)
    listed = DENSE + SHORT + GROUPED
    want = [c[0] for c in listed]
    wrong = [(c, g) for c, g, w in zip(listed, got, want) if g != w]
    assert len(got) == len(want) and not wrong


def test_the_list_covers_every_kernel():
    seen = set()
    for rows, fmt, _, N, K in DENSE:
        seen |= {("dense", rows, fmt, "aligned", K % 256 == 0), ("dense", rows, fmt, "pieces", N % 16 == 0)}
    for rows, fmt, _, _, N, K in GROUPED:
        seen |= {("grouped", rows, fmt, "aligned", K % 256 == 0), ("grouped", rows, fmt, "pieces", N % 16 == 0)}
    assert seen == {(kind, rows, fmt, what, yes) for kind in ("dense", "grouped") for rows in (16, 32, 64, 128, 256)
                    for fmt in ("nv", "mx") for what in ("aligned", "pieces") for yes in (True, False)}
    assert any(tail for _, _, _, tail, _, _ in GROUPED) and any(0 in s for _, _, s, _, _, _ in GROUPED)


def test_choice_at_the_ends(choose):
    """Empty contractions, one row, and sizes past any card: always one of the five."""
    big = 1 << 30
    cases = [(mx, g, M, N, K, cus) for mx in (0, 1) for g in (0, 1, 1 << 20) for M in (1, big) for N in (1, big)
             for K in (0, 32, (1 << 23) - 32) for cus in (1, 256)]
    got = choose(cases)
    assert set(got) <= {16, 32, 64, 128, 256}
    for (mx, g, M, N, K, _), rows in zip(cases, got):
        assert rows == 256 or K > 0
        assert rows != 128 or (M // 128 + min(g, M)) * -(-N // 128) < 1 << 31
