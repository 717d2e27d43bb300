"""The work line of 4-bit chunk attention (csrc/attend_plan.h) replayed on the host
(helpers/attend4_plan_replay.cpp), cut into spans with a charge per group, or group by group into pieces:
every key step of every row tile is computed by exactly one workgroup, and the join reads the records
that were written and no others."""
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "draft_sampling_verification_w1_amd", "csrc")
TILES = (16, 32, 48, 64, 96, 128, 192, 256, 384)


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path_factory.mktemp("plan4") / "replay")
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-I", CSRC, "-o", exe,
                           os.path.join(HERE, "helpers", "attend4_plan_replay.cpp")])

    def run(calls):
        """calls: (grid, rows, group, kv_heads, width, extra, [(cached, chunk) per slot]); how many were cut by group"""
        text = "".join(f"{g} {r} {q} {h} {w} {e} {len(s)} " + " ".join(f"{a} {b}" for a, b in s) + "\n"
                       for g, r, q, h, w, e, s in calls)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(calls)
        wrong = [(c, g) for c, g in zip(calls, got) if g[:3] != (0, 0, 0)]
        assert not wrong, (len(wrong), wrong[0])
        return sum(g[3] for g in got)
    return run


@pytest.mark.parametrize("extra", [0, 1, 20])
def test_random_batches(replay, extra):
    rng = random.Random(12 + extra)
    calls = []
    for _ in range(3000):
        rows, group = rng.choice(TILES), rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16, 64])
        most = max(2, 8 * rows // group)
        slots = [(rng.choice([0, rng.randrange(100), rng.randrange(4000)]),
                  rng.choice([0, 1, rng.randrange(most), rows // group * rng.randrange(1, 8) + rng.randrange(2)]))
                 for _ in range(rng.randrange(1, 12))]
        width = rng.choice([1 << 20, 1 << 20, 16 * rng.randrange(1, 300)])
        calls.append((rng.choice([256, 512, 8]), rows, group, rng.randrange(1, 4), width, extra, slots))
    replay(calls)


def test_groups_cut_by_themselves(replay):
    rng = random.Random(3)
    calls = [(rng.choice([256, 512]), 96, 4, rng.choice([1, 2, 8]), 1 << 20, 0,
              [(rng.choice([0, 5, rng.randrange(30000)]), rng.choice([0, 1, rng.randrange(18)]))
               for _ in range(rng.randrange(1, 17))]) for _ in range(3000)]
    cut = replay(calls)
    assert cut > 2500


@pytest.mark.parametrize("grid,heads,slots", [(512, 8, [(30000, 1)]), (512, 1, [(0, 1)]), (256, 128, [(100, 1)]),
                                              (256, 1, [(7, 1)] * 128), (256, 1, [(7, 1)] * 129), (512, 2, [(0, 0)] * 5)])
def test_edges(replay, grid, heads, slots):
    replay([(grid, rows, 4, heads, 1 << 20, 0, slots) for rows in TILES])
