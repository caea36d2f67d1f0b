"""Which copies a kernel with a ring of stages still has to wait for when a wait of its own ran out: the
count of copies into each stage (tc_util.cuh's ring_fills, compiled for the host) against the ring played
through step by step, for every step at which the wait may run out."""
import subprocess

import pytest

PROGRAM = r"""
#include <cstdio>
#include "tc_util.cuh"
int main() {
    for (int stages = 1; stages <= 8; ++stages)
        for (int loads = 0; loads <= 40; ++loads)
            for (int s = 0; s < stages; ++s)
                printf("%d %d %d %d\n", stages, loads, s, kda::tc::ring_fills(loads, s, stages));
}
"""


@pytest.fixture(scope="module")
def fills(tmp_path_factory):
    from serving_kda_chunkwise_gb300 import build
    at = tmp_path_factory.mktemp("ring")
    src, exe = at / "ring.cu", at / "ring"
    src.write_text(PROGRAM)
    subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-I", build.INCLUDE, "-I", build.CSRC,
                    "-o", str(exe), str(src)], check=True, capture_output=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    rows = [tuple(map(int, line.split())) for line in out.splitlines()]
    return {r[:3]: r[3] for r in rows}


def _play(rows, stages, ahead, runs_out):
    """(copies started, their stages in turn, rows that were waited for) of a ring that starts `ahead`
    copies before the first row and one more in every row after the wait of that row."""
    started, waited = [], 0
    for r in range(min(ahead, rows)):
        started.append(r % stages)
    for r in range(rows):
        if r == runs_out:
            break
        waited += 1
        if len(started) < rows and (ahead == stages - 1 or stages == 1 or r > 0):
            started.append(len(started) % stages)
    return started, waited


@pytest.mark.parametrize("stages", range(1, 9))
def test_every_copy_on_its_way_is_waited_for(fills, stages):
    for ahead in {max(stages - 1, 1), stages}:
        for rows in range(0, 30):
            for runs_out in range(rows):
                started, waited = _play(rows, stages, ahead, runs_out)
                assert len(started) <= 40
                for s in range(stages):
                    mine = [k for k, at in enumerate(started) if at == s]
                    n = fills[stages, len(started), s]
                    assert n == len(mine)
                    # one copy of a stage at most is not waited for yet, the last: its phase's parity
                    late = [k for k in mine if k >= waited]
                    assert len(late) <= 1 and late == mine[len(mine) - len(late):]


@pytest.mark.parametrize("stages,ahead", [(2, 2), (3, 2)])
def test_fills_of_a_scan_that_leaves_its_steps(fills, stages, ahead):
    """The scans of the channel recurrence fill a stage behind the barrier of every step that they stay
    in; one that leaves at step k has started min(k + ahead, its tiles) fills.  All of those whose phase
    no step before k has seen end are the last ones of their stages, and no stage has two."""
    for tiles in range(0, 30):
        for steps in range(tiles, tiles + 2):  # (a step at the end may have no tile for this CTA)
            for k in range(steps + 1):
                started = list(range(min(ahead, tiles)))
                for step in range(k):
                    if step + ahead < tiles:
                        started.append(step + ahead)
                loads = min(k + ahead, tiles)
                assert started == list(range(loads))
                for s in range(stages):
                    mine = [t for t in started if t % stages == s]
                    late = [t for t in mine if t >= k]
                    assert fills[stages, loads, s] == len(mine)
                    assert len(late) <= 1 and late == mine[len(mine) - len(late):]
