"""The ring of rows of the residual RMS norm's backward, without a GPU: its layout over all widths, from the same host
code that the launcher uses, against what one-bit phase parities need.

A team that waits for a group of rows while the slot's previous group has not landed takes the wrong phase for its own
(the barrier's parity is one bit).  It has waited for that group only if it had a row in it, so every team with a row in
a group must have one in the group that the slot held before."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_transformer_mlp_tp_gb300", "csrc")
SMEM, MAX_SLOTS = 196608, 32

PROGRAM = r"""
#include <stdio.h>
#include "bwd_ring.h"

int main(int argc, char**) {
  int rows, d, sms, teams;
  if (argc > 1) {
    while (scanf("%d %d %d %d", &rows, &d, &sms, &teams) == 4)  // groups, group, slots, teams
      printf("%d\n", tpmlp::bwd_ring_ok(rows, d, sms, teams) ? 1 : 0);
    return 0;
  }
  while (scanf("%d %d %d", &rows, &d, &sms) == 3) {
    const tpmlp::BwdRing r = tpmlp::bwd_ring(rows, d, sms);
    printf("%d %d %d %d %d %d %d %d %d %d\n", r.blocks, r.vt, r.team_warps, r.teams, r.group, r.slots, r.most,
           r.slot_bytes, r.smem, tpmlp::bwd_ring_ok(r.most, r.group, r.slots, r.teams) ? 1 : 0);
  }
  return 0;
}
"""
FIELDS = ("blocks", "vt", "team_warps", "teams", "group", "slots", "most", "slot_bytes", "smem", "ok")


@pytest.fixture(scope="module")
def layouts(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    tmp = tmp_path_factory.mktemp("ring")
    (tmp / "ring.cpp").write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(tmp / "ring.cpp"), "-o", str(tmp / "ring")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(cases, *mode):
        out = subprocess.run([str(tmp / "ring"), *mode], input="".join(" ".join(map(str, c)) + "\n" for c in cases),
                             capture_output=True, text=True, timeout=60).stdout.split("\n")
        return [dict(zip(("ok",) if mode else FIELDS, map(int, line.split()))) for line in out if line]

    return run


def teams_of(group, i, teams):
    """Teams with a row in the block's group i (a whole one)."""
    return {n % teams for n in range(i * group, i * group + min(group, teams))}


def parity_safe(groups, group, slots, teams):
    # the pattern of teams repeats after `teams` groups
    return all(teams_of(group, i, teams) <= teams_of(group, i - slots, teams)
               for i in range(slots, min(groups, slots + teams)))


@pytest.mark.parametrize("rows", [1, 7, 152, 153, 1369, 1673, 5473, 8192, 70001, 1 << 20, (1 << 30) - 1])
def test_every_team_of_a_group_knows_the_slots_previous_group(layouts, rows):
    cases = [(rows, d, sms) for d in range(8, 16392, 8) for sms in (152, 148, 20, 1)]
    bad = []
    for case, r in zip(cases, layouts(cases)):
        assert r["group"] >= 1 and 1 <= r["slots"] <= MAX_SLOTS and r["slots"] <= r["most"]
        assert r["slot_bytes"] == 6 * case[1] * r["group"] and r["slots"] * r["slot_bytes"] <= r["smem"] <= SMEM
        assert r["teams"] * r["team_warps"] == 16 and r["team_warps"] * r["vt"] * 256 >= case[1]
        assert r["blocks"] * r["most"] * r["group"] >= rows > (r["most"] - 1) * r["group"] * r["blocks"]
        assert r["smem"] >= 4 * r["teams"] * case[1]
        safe = parity_safe(r["most"], r["group"], r["slots"], r["teams"])
        if not safe or not r["ok"]:
            bad.append((case, r))
    assert not bad, f"{len(bad)} layouts, the first {bad[0]}"


def test_the_launchers_own_check_agrees(layouts):
    """bwd_ring_ok, which the launcher asks before it launches, against the condition itself."""
    cases = [(groups, group, slots, teams) for teams in (1, 2, 4, 8, 16) for group in range(1, 20)
             for slots in range(1, 33) for groups in (slots, slots + 1, 10 * slots + teams)]
    for case, r in zip(cases, layouts(cases, "check")):
        groups, group, slots, teams = case
        if groups == slots + 1:  # one turn more: the check may refuse what this count alone would allow
            assert not r["ok"] or parity_safe(*case)
        else:
            assert bool(r["ok"]) == parity_safe(*case), case
    assert not any(r["ok"] for r in layouts([(9, 0, 4, 1), (9, 4, 0, 1), (9, 16, 33, 1), (9, 16, 33, 16)], "check"))


def test_rings_keep_most_of_the_shared_memory(layouts):
    """Rounding for the parities leaves rings of long inputs at least four fifths full where rows are short."""
    cases = [(1 << 20, d, 152) for d in range(8, 4104, 8)]
    for case, r in zip(cases, layouts(cases)):
        assert r["slots"] * r["slot_bytes"] >= 0.8 * min(SMEM, MAX_SLOTS * r["slot_bytes"]), (case, r)
