"""What a slot may write belongs to it alone: the rule of the paged cache's tables that
keeps one slot's tokens out of another's, on the plain model (cache_model.py) that the GPU
tests compare the tables with."""
import random

import pytest

from cache_model import CacheModel


def check_writers(lens, rows, page, add, status):
    """After a reserve: every page that an accepted slot is about to write is held by no
    other slot, or only by slots whose tokens end before it writes and that do not write
    there themselves."""
    users = {}
    for s, row in enumerate(rows):
        for j, p in enumerate(row):
            users.setdefault(p, []).append((s, j))
    for s, n in enumerate(add):
        if n <= 0 or status[s] != 0:
            continue
        assert len(rows[s]) * page >= lens[s] + n
        for j in range(lens[s] // page, (lens[s] + n - 1) // page + 1):
            start = max(lens[s] - j * page, 0)  # first position that it writes in this page
            for other, i in users[rows[s][j]]:
                if other == s:
                    continue
                assert (add[other] <= 0 or status[other] != 0) or i < lens[other] // page, (s, other, j)
                assert lens[other] - i * page <= start, (s, other, j)


@pytest.mark.parametrize("lens,reserved", [(16, 5), (0, 5), (0, 40), (7, 40), (32, 33), (16, 17)])
def test_fork_of_reserved_pages(lens, reserved):
    """Pages that are reserved and hold no token are not shared by a fork."""
    m = CacheModel(3, 8, 30, 16)
    assert m.reserve([lens, 0, 0])[0] == [0, 0, 0]
    m.commit([lens, 0, 0], 0)
    assert m.reserve([reserved, 0, 0])[0] == [0, 0, 0]
    assert m.fork([0], [1]) == [0]
    assert m.lens[1] == lens and len(m.rows[1]) == -(-lens // 16)
    for add in ([reserved, reserved, 0], [1, 1, 0], [0, 17, 0]):
        st = m.reserve(add)[0]
        assert st == [0, 0, 0]
        check_writers(m.lens, m.rows, 16, add, st)


@pytest.mark.parametrize("seed", range(6))
def test_random_calls(seed):
    rng = random.Random(seed)
    slots, page = rng.randint(2, 12), 16
    m = CacheModel(slots, rng.randint(2, 6), rng.randint(6, 40), page)
    for _ in range(400):
        op = rng.choice(["reserve", "reserve", "fork", "fork", "commit", "rollback", "free", "compact"])
        if op == "reserve":
            add = [rng.choice([0, 1, rng.randint(1, 40)]) for _ in range(slots)]
            st = m.reserve(add)[0]
            check_writers(m.lens, m.rows, page, add, st)
            if rng.random() < 0.5:
                m.commit([rng.randint(0, a) if st[s] == 0 else -2 ** 31 for s, a in enumerate(add)], 0)
        elif op == "fork":
            m.fork([rng.randrange(slots)], [rng.randrange(slots)])
        elif op == "commit":
            # a slot's tokens end where it was told to write at most
            m.commit([0] * slots, 0)
        elif op == "rollback":
            m.commit([-rng.choice([0, 1, 5, 40]) for _ in range(slots)], 0)
        elif op == "free":
            m.free([rng.randrange(slots)])
        else:
            m.compact()
