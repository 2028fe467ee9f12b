"""The runs of dW's tiles that single CTAs take (csrc/ce_runs.h), compiled for
the host: they tile the launch exactly, whatever the sizes, and stay balanced."""

import os
import shutil
import subprocess

import pytest

from block_sparse_long_bwd_b200 import binding as bb

CSRC = os.path.join(os.path.dirname(bb.LIB_PATH), "csrc")
MAIN = r"""
#include <stdio.h>
#include "ce_runs.h"
int main() {
  int wm, dn, cols, ch, cw, workers, start[1025];
  long long nh;
  while (scanf("%d %d %d %lld %d %d %d", &wm, &dn, &cols, &nh, &ch, &cw, &workers) == 7) {
    bb::dw_runs(wm, dn, cols, nh, ch, cw, workers, start);
    for (int w = 0; w <= workers; ++w) printf("%d ", start[w]);
    printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def runs(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("runs")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover", "-I", CSRC, str(d / "main.cpp"), "-o",
                    str(d / "runs")], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(d / "runs")], input=text, capture_output=True, text=True,
                             check=True).stdout
        return [list(map(int, line.split())) for line in out.splitlines()]

    return run


def _case(hidden, V, splits, sms=148):
    """The arguments of a launch over V words: 128 x 256 tiles, 64-wide K steps."""
    dn, wm, cols = -(-hidden // 256), -(-V // 128), -(-hidden // 64)
    nh = dn * splits
    ch = max(4, -(-V // 64) // splits)
    return wm, dn, cols, nh, ch, 4, min(nh + wm * dn, sms)


def _cases():
    for hidden in (64, 72, 256, 264, 320, 768, 776, 1024, 1536, 8192, 65536):
        for V in list(range(1, 700, 23)) + [1000, 3001, 6417, 30011, 50021, 524288, 1 << 20]:
            for splits in (1, 2, 3, 8, 24, 64):
                if splits == 1 or -(-V // 64) // splits >= 4:
                    yield _case(hidden, V, splits)
    yield _case(768, 5000, 4, sms=1)
    yield _case(768, 5000, 4, sms=7)


def test_runs_tile_the_launch(runs):
    cases = list(_cases())
    got = runs(cases)
    assert len(got) == len(cases)
    for c, start in zip(cases, got):
        wm, dn, workers = c[0], c[1], c[6]
        assert len(start) == workers + 1
        assert start[0] == 0 and start[-1] == wm * dn, c
        assert all(a <= b for a, b in zip(start, start[1:])), c


def test_runs_are_balanced(runs):
    """Costs in K steps (a tile of dW: cw per 5 units of its blocks plus one):
    no worker is above the mean share by more than one tile of dh and two of dW."""
    for c, start in zip(cases := list(_cases()), runs(cases)):
        wm, dn, cols, nh, ch, cw, workers = c
        unit = [(min(4, cols - 4 * n) + 1) * cw / 5 for n in range(dn)]
        cum = [0.0]
        for n in range(dn):
            cum.append(cum[-1] + unit[n] * wm)

        def upto(t):
            n = min(t // wm, dn - 1)
            return cum[n] + (t - n * wm) * unit[n]

        load = [upto(start[w + 1]) - upto(start[w]) + ch * (nh // workers + (w < nh % workers))
                for w in range(workers)]
        assert max(load) <= sum(load) / workers + ch + 2 * cw, c
