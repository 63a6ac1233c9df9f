"""How a product of up to eight tokens with 4-bit weights is split over blocks, without a GPU: from the same host code that the
launcher uses, what a block keeps in shared memory against what it has, over the sizes that the calls take."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_transformer_mlp_tp_gb300", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include "few_plan_w4.h"

int main() {
  int M, N, K, mats, g32, zeros, fit1, fit2, fit4;
  while (scanf("%d %d %d %d %d %d %d %d %d", &M, &N, &K, &mats, &g32, &zeros, &fit1, &fit2, &fit4) == 9) {
    const int fixed = tpmlp::w4_few_fixed(g32 != 0, zeros != 0);
    const tpmlp::W4FewPlan p =
        tpmlp::w4_few_plan(M, N, K, mats, fixed, [&](int r) { return r == 1 ? fit1 : r == 2 ? fit2 : fit4; });
    printf("%d %d %d %d %d %d %d %d\n", p.ranks, p.clusters, p.chunk, p.stages, p.round, p.x_pitch, fixed,
           tpmlp::kW4FewSmem);
  }
  return 0;
}
"""
FIELDS = ("ranks", "clusters", "chunk", "stages", "round", "x_pitch", "fixed", "smem")
TEAMS, SUMS = 2, 8 * 8 * 16 * 4  # a column tile's sums: warps of a team x tokens x columns, fp32
LARGEST = (2 ** 31 - 1) // 2 // 8 * 8  # of N and K


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    tmp = tmp_path_factory.mktemp("plan")
    (tmp / "plan.cpp").write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(tmp / "plan.cpp"), "-o", str(tmp / "plan")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(cases):
        out = subprocess.run([str(tmp / "plan")], input="".join(" ".join(map(str, c)) + "\n" for c in cases),
                             capture_output=True, text=True, timeout=60).stdout.split("\n")
        out = [dict(zip(FIELDS, map(int, line.split()))) for line in out if line]
        assert len(out) == len(cases)
        return out

    return run


def room_for_x(M, K, ranks, fixed, smem):
    """Bytes that a block of `ranks` has beside its part of X and what it always keeps."""
    tiles = (K + 63) // 64
    return smem - fixed - M * ((tiles + ranks - 1) // ranks * 128 + 16)


@pytest.mark.parametrize("K", [8, 64, 200, 1024, 4096, 4104, 16384, 40000, 65544, 131072, 210000, 524296, 1 << 20, 1 << 24,
                               1 << 28, (1 << 29) - 8, 1 << 29, (1 << 29) + 8, LARGEST - 1048, LARGEST - 56, LARGEST - 48, LARGEST])
def test_a_block_keeps_no_more_than_its_shared_memory(plans, K):
    fits = ((152, 76, 32), (148, 70, 30), (20, 10, 4), (1, 1, 1))
    cases = [(M, N, K, mats, g32, zeros, *fit) for M in range(1, 9) for N in (8, 16, 24, 4096, 16384, 139272, LARGEST)
             for mats in (1, 2) for g32 in (0, 1) for zeros in (0, 1) for fit in fits]
    k_tiles = (K + 63) // 64
    for case, p in zip(cases, plans(cases)):
        M, N, _, mats, _, _, *fit = case
        if p["clusters"] == 0:  # no split has room for X, 32 KB of codes in flight and two tiles' sums
            least = max(room_for_x(M, K, r, p["fixed"], p["smem"]) for r in (1, 2, 4) if r <= k_tiles)
            assert least < 32768 + 2 * SUMS, (case, p)
            continue
        mine = (k_tiles + p["ranks"] - 1) // p["ranks"]
        assert p["ranks"] in (1, 2, 4) and p["ranks"] <= k_tiles, (case, p)
        assert 1 <= p["clusters"] <= max(fit) and p["clusters"] <= (N + 15) // 16, (case, p)
        assert p["x_pitch"] == mine * 128 + 16, (case, p)
        assert 1 <= p["chunk"] <= 64 and 1 <= p["stages"] <= 4, (case, p)
        assert p["round"] >= mats and p["round"] % mats == 0, (case, p)
        # barriers and the abort flag: the last 256 bytes of what is always kept
        assert 2 * 8 * TEAMS * p["stages"] + 4 <= 256, (case, p)
        used = TEAMS * p["stages"] * p["chunk"] * 512 + p["round"] * SUMS + M * p["x_pitch"] + p["fixed"]
        assert used <= p["smem"], (case, p)
