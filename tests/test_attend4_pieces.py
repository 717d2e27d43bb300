"""The cut of few groups into pieces (csrc/attend_plan.h) replayed on the host by the functions that the kernel calls
(helpers/attend4_pieces_replay.cpp): the packed sums, the choice among the targets and the look-up of a workgroup's
piece, with slots without tokens in front, between and behind."""
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "draft_sampling_verification_w1_amd", "csrc")


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path_factory.mktemp("pieces") / "replay")
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, "-o", exe,
                           os.path.join(HERE, "helpers", "attend4_pieces_replay.cpp")])

    def run(calls):
        """calls: (grid, rows, group, kv_heads, width, [(cached, chunk) per slot]); the numbers of pieces"""
        text = "".join(f"{g} {r} {q} {h} {w} {len(s)} " + " ".join(f"{a} {b}" for a, b in s) + "\n"
                       for g, r, q, h, w, s in calls)
        got = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        got = [tuple(map(int, line.split())) for line in got]
        assert len(got) == len(calls)
        for c, (pieces, *wrong) in zip(calls, got):
            assert wrong == [0, 0, 0] and 1 <= pieces <= c[0], (c, pieces, wrong)
        return [g[0] for g in got]
    return run


def test_random_batches(replay):
    rng = random.Random(5)
    calls = []
    while len(calls) < 4000:
        grid, heads = rng.choice([256, 512]), rng.choice([1, 2, 3, 8, 16])
        slots = [(rng.choice([0, rng.randrange(40), rng.randrange(3000), rng.randrange(200000)]),
                  rng.choice([0, 0, 1, rng.randrange(1, 18)])) for _ in range(rng.randrange(1, grid // (2 * heads) + 1))]
        if any(c for _, c in slots):
            calls.append((grid, 96, rng.choice([1, 2, 4, 5]), heads, rng.choice([1 << 20, 1 << 20, 16 * rng.randrange(1, 400)]),
                          slots))
    replay(calls)


@pytest.mark.parametrize("grid", [256, 512])
def test_most_and_fewest(replay, grid):
    full = [(grid, 16, 4, 1, 1 << 28, [(n, 1)] * (grid // 2)) for n in (0, 31, 1000, 1 << 20)]
    lone = [(grid, 16, 4, heads, 1 << 28, [(0, 0)] * before + [(n, 1)] + [(5, 0)] * behind)
            for heads in (1, 2) for n in (0, 100, 30000, (1 << 28) - 2)
            for before, behind in ((0, 0), (grid // 4 - 1, 0), (0, grid // 4 - 1), (17, 40))]
    assert min(replay(full)) == grid // 2
    replay(lone)
