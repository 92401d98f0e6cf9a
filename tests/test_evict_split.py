"""How an eviction is split over blocks: by the device's SMs (CPU only)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "split_w4a16_quantized_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "qmm_evict_split.h"
int main() {
    long long columns;
    int cap, keep, lanes, sms;
    while (std::scanf("%lld %d %d %d %d", &columns, &cap, &keep, &lanes, &sms) == 5) {
        const qmm::EvictSplit s = qmm::evict_split(columns, cap, keep, lanes, sms);
        std::printf("%d %d %d %d %d %d\n", s.slices, s.lanes, s.movers, s.cluster, s.spread, s.held);
    }
}
"""

CASES = [(columns, cap, keep, lanes) for columns in (1, 8, 36, 75, 76, 151, 152, 288, 303, 304, 1536, 70000)
         for cap in (8, 1152, 7008, 16384, 16385, 100000, 131072, 1 << 24)
         for keep in (1, 256, 257, 16384) if keep <= cap for lanes in (4, 8, 16)]


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    at = tmp_path_factory.mktemp("split")
    src, exe = at / "split.cpp", at / "split"
    src.write_text(PROGRAM)
    subprocess.run([shutil.which("g++"), "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)

    def ask(cases):
        said = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, c)) for c in cases),
                              check=True, capture_output=True, text=True).stdout
        return [tuple(map(int, line.split())) for line in said.splitlines()]
    return ask


@pytest.mark.parametrize("sms", [1, 20, 76, 132, 152, 200])
def test_split_follows_the_sms(split, sms):
    """Whole rows and a block a column where those fill the SMs; else no more pieces and
    blocks than fill them, and no column without room for its slots but those longer than
    all of its blocks hold."""
    for (columns, cap, keep, row), (slices, lanes, movers, cluster, spread, held) in zip(
            CASES, split([(*c, sms) for c in CASES])):
        at = (columns, cap, keep, row, sms)
        assert slices * lanes == row and lanes >= 4, at
        pools = 2 * columns
        assert slices == 1 or pools * slices // 2 < 4 * sms, at
        assert pools * slices >= 4 * sms or lanes == 4, at
        assert movers == 1 or (lanes == 4 and pools * slices * movers // 2 < 2 * sms and
                               2 * keep // movers > 256), at
        need = 1
        while need < 8 and -(-cap // need) > 16384:
            need *= 2
        assert cluster >= need and cluster in (1, 2, 4, 8), at
        assert cluster == need or columns * cluster // 2 < sms, at
        assert cluster == 8 or columns * cluster >= sms or cap // cluster <= 2048, at
        if cluster > 1:
            assert spread == (cluster > need or columns * cluster <= 2 * sms), at
        assert held % 64 == 0 and held <= 16384, at
        assert held * cluster >= cap or (cluster == 8 and held == 16384), at


def test_no_rule_counts_the_sms_of_one_chip():
    for name in ("qmm_evict.cu", "qmm_evict_split.h", "qmm_prefix_attention.cu",
                 "qmm_scored_attention.cu", "qmm_mass_tc.cu"):
        code = [line.split("//")[0] for line in open(os.path.join(CSRC, name))]
        assert not any("152" in line for line in code), name
