"""How many threads the gradient of combine gives a token (host arithmetic, compiled
from csrc/dg_rows.h; no GPU): by the SMs of the device that it runs on."""
import os
import shutil
import subprocess

import pytest

from moe_grouped_gemm_bf16_gb300 import _build

SOURCE = """
#include <cstdio>
#include <cstdlib>
#include "dg_rows.h"
int main(int argc, char** argv) {
  for (int i = 1; i + 4 < argc; i += 5) {
    const int T = std::atoi(argv[i]), K = std::atoi(argv[i + 1]), k = std::atoi(argv[i + 2]);
    std::printf("%d\\n", dgk::combine_team(T, K / 8, k, std::atoi(argv[i + 3]), std::atoi(argv[i + 4])));
  }
}
"""


@pytest.fixture(scope="module")
def team(tmp_path_factory):
    at = tmp_path_factory.mktemp("team")
    (at / "team.cpp").write_text(SOURCE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-I", _build.CSRC, "-I", cuda, str(at / "team.cpp"),
                    "-o", str(at / "team")], check=True)

    def of(*calls):
        out = subprocess.run([str(at / "team"), *(str(v) for c in calls for v in c)], check=True, capture_output=True,
                             text=True)
        return [int(v) for v in out.stdout.split()]
    return of


def rows_of(k):
    return 2 if k <= 2 else 4 if k <= 4 else 8


def by_hand(T, K, k, sms):
    """The team with the fewest rounds times (1 + its loads of a round), the larger of equal ones."""
    vecs, rows = K // 8, rows_of(k)

    def cost(n):
        at_once = sms * 3 * 256 // n
        return -(-T // at_once) * (1 + -(-vecs // (n * (8 // rows))) * -(-k // rows))
    return min((256, 128, 64, 32), key=cost)


def test_teams_go_by_the_devices_sms(team):
    calls = [(T, K, k, sms) for T in (1, 40, 300, 480, 700, 1365, 4096, 9451) for K in (8, 360, 2048, 7168, 16384)
             for k in (1, 3, 8, 9) for sms in (152, 76, 132, 20, 1)]
    got = team(*((T, K, k, rows_of(k), sms) for T, K, k, sms in calls))
    assert got == [by_hand(*c) for c in calls]
    # (the device's number of SMs does change the choice)
    assert any(by_hand(T, K, k, 152) != by_hand(T, K, k, sms) for T, K, k, sms in calls)


def test_teams_of_152_sms_stay(team):
    assert team((9451, 360, 1, 2, 152), (480, 7688, 8, 8, 152), (4096, 7168, 8, 8, 152)) == [32, 128, 128]
