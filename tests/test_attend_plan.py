"""The work line of chunk attention (csrc/attend_plan.h), replayed on the host
(helpers/attend_plan_replay.cpp): every key step of every row tile is computed by exactly
one workgroup, and no joined group reaches behind the last span."""
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "draft_sampling_verification_w1_amd", "csrc")
TILES = (16, 32, 64, 96, 128, 192, 256, 384)


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path_factory.mktemp("plan") / "replay")
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-I", CSRC, "-o", exe,
                           os.path.join(HERE, "helpers", "attend_plan_replay.cpp")])

    def run(calls):
        """calls: (grid, rows, group, kv_heads, width, [(cached, chunk) per slot])"""
        text = "".join(f"{g} {r} {q} {h} {w} {len(s)} " + " ".join(f"{a} {b}" for a, b in s) + "\n"
                       for g, r, q, h, w, s in calls)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(calls)
        wrong = [(c, g) for c, g in zip(calls, got) if g != (0, 0, 0)]
        assert not wrong, (len(wrong), wrong[0])
    return run


@pytest.mark.parametrize("grid,rows,group,kv_heads,slots", [
    (256, 384, 1, 2, [(0, 1153)]),             # an almost empty last tile
    (256, 384, 4, 8, [(30, 290)]),
    (256, 384, 1, 16, [(2000, 1200)]),
    (256, 384, 1, 16, [(2000, 1200), (5, 3), (0, 1153)]),
    (256, 128, 1, 1, [(0, 385)]),
    (512, 96, 1, 3, [(7, 289), (0, 290)]),
])
def test_short_last_tile(replay, grid, rows, group, kv_heads, slots):
    replay([(grid, rows, group, kv_heads, 1 << 20, slots)])


def test_table_shorter_than_the_chunk(replay):
    """Tokens that the table has no place for are dropped; the others' steps are all there."""
    replay([(256, rows, group, 2, width, [(cached, 2048), (0, 40)])
            for rows in TILES for group in (1, 3) for width in (16, 64, 1024) for cached in (0, 9, 1024, 5000)])


def test_random_batches(replay):
    rng = random.Random(11)
    calls = []
    for _ in range(4000):
        rows = rng.choice(TILES)
        group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16, 64])
        most = max(2, 8 * rows // group)
        slots = [(rng.choice([0, rng.randrange(100), rng.randrange(4000)]),
                  rng.choice([0, 1, rng.randrange(most), rows // group * rng.randrange(1, 8) + rng.randrange(2)]))
                 for _ in range(rng.randrange(1, 6))]
        width = rng.choice([1 << 20, 1 << 20, 16 * rng.randrange(1, 300)])
        calls.append((rng.choice([256, 512, 8]), rows, group, rng.randrange(1, 4), width, slots))
    replay(calls)
