"""Forks of slots that hold reserved pages without tokens: tables against the plain model,
and what each slot then finds on its pages."""
import random

import numpy as np
import pytest

from cache_model import CacheModel
from test_cache_ownership import check_writers
from test_gpu_cache import C, ints, same  # noqa: F401

pytestmark = pytest.mark.gpu


def tokens(c, s, n):
    """The first n tokens' keys and values of a slot with one head, [n, head_dim] each."""
    page, rows = c.page_size, c.table[s].cpu()
    e = 16 // c.dtype.itemsize
    K = [c.K[0, int(rows[p // page]), 0, :, p % page, :].reshape(-1) for p in range(n)]
    V = [c.V[0, int(rows[p // page]), 0, p % page // e, :, p % page % e] for p in range(n)]
    return [k.tolist() for k in K], [v.tolist() for v in V]


@pytest.mark.parametrize("lens,reserved,add", [
    (16, 5, (1, 1)), (16, 17, (17, 17)), (0, 5, (5, 5)), (0, 40, (3, 20)), (7, 40, (40, 40)), (7, 9, (0, 12)),
    (32, 33, (20, 33)), (31, 2, (2, 1))])
def test_fork_of_reserved_pages(C, lens, reserved, add):  # noqa: F811
    """Both continuations of a slot write different tokens; each finds its own."""
    import torch
    m = CacheModel(3, 8, 30, 16)
    c = C.PagedCache(3, 8, 30, 16, 1, 1, 64, torch.float32)
    for rows in ([lens, 0, 0], [reserved, 0, 0]):
        assert c.reserve(ints(rows))["status"].tolist() == m.reserve(rows)[0] == [0, 0, 0]
        if rows[0] == lens:
            old = torch.arange(max(1, lens), device="cuda").view(-1, 1, 1).expand(-1, 1, 64).float().contiguous()
            c.append(0, old, old, ints([0, lens, lens, lens]))
            c.commit(ints(rows))
            m.commit(rows, 0)
    assert c.fork(ints([0]), ints([1])).tolist() == m.fork([0], [1]) == [0]
    same(c, m, "fork")
    both = list(add) + [0]
    assert c.reserve(ints(both))["status"].tolist() == m.reserve(both)[0] == [0, 0, 0]
    same(c, m, "reserve")
    check_writers(m.lens, m.rows, 16, both, [0, 0, 0])
    new = torch.cat([torch.full((add[s], 1, 64), 1000.0 * (s + 1), device="cuda") +
                     torch.arange(add[s], device="cuda").view(-1, 1, 1) for s in range(2)])
    c.append(0, new, new, ints([0, add[0], sum(add), sum(add)]))
    c.commit(ints(both))
    for s in range(2):
        want = [[float(p)] * 64 for p in range(lens)] + [[1000.0 * (s + 1) + i] * 64 for i in range(add[s])]
        K, V = tokens(c, s, lens + add[s])
        assert K == want and V == want, s


@pytest.mark.parametrize("slots,max_pages,pages", [(5, 6, 20), (12, 4, 30), (40, 5, 400)])
def test_writers_own_their_pages(C, slots, max_pages, pages):  # noqa: F811
    """Random calls, many of them forks of slots with reserved pages: after every reserve
    the pages that a slot may write are its own, and the counts are those of the tables."""
    rng = random.Random(slots)
    m, c = CacheModel(slots, max_pages, pages, 16), C.PagedCache(slots, max_pages, pages, 16, 1, 1, 64)
    for step in range(60):
        op = rng.choice(["reserve", "reserve", "fork", "fork", "commit", "free"])
        if op == "reserve":
            add = [rng.choice([0, 1, rng.randint(1, 40)]) for _ in range(slots)]
            got = c.reserve(ints(add))["status"].tolist()
            assert got == m.reserve(add)[0]
            rows = [[p for p in r if p >= 0] for r in c.table.tolist()]
            check_writers(c.lens.tolist(), rows, 16, add, got)
            if rng.random() < 0.5:
                keep = [rng.randint(0, a) if got[s] == 0 else -2 ** 31 for s, a in enumerate(add)]
                c.commit(ints(keep))
                m.commit(keep, 0)
        elif op == "fork":
            src, dst = [rng.randrange(slots) for _ in range(3)], [rng.randrange(slots) for _ in range(3)]
            assert c.fork(ints(src), ints(dst)).tolist() == m.fork(src, dst)
        elif op == "commit":
            keep = [-rng.choice([0, 0, 1, 5, 40]) for _ in range(slots)]
            c.commit(ints(keep))
            m.commit(keep, 0)
        else:
            gone = [rng.randrange(slots)]
            c.free(ints(gone))
            m.free(gone)
        same(c, m, f"step {step} {op}")
        table, held = c.table.cpu().numpy(), c.held.cpu().numpy()
        inside = np.arange(max_pages)[None] < held[:, None]
        refs = np.bincount(table[inside], minlength=pages)
        np.testing.assert_array_equal(c.refs.cpu().numpy(), refs)
        free = np.unpackbits(c.free_bits.cpu().numpy().view(np.uint8), bitorder="little")[:pages]
        np.testing.assert_array_equal(free, refs == 0)
        assert c.n_free.item() == free.sum()


def test_round_repeated_after_a_fork(C):  # noqa: F811
    """A round of the decoding loop that ends for want of pages leaves the served requests'
    pages reserved; a request is forked before the round is repeated, and both attend over
    their own tokens (Target.forward checks every attended row)."""
    from draft_sampling_verification_w1_amd import dspark
    import test_gpu_serving as S
    t = S.Target(dspark, "bf16", max_pages=4, pages=12)
    rng = np.random.default_rng(3)
    t.prompt([rng.integers(0, S.V, n).tolist() for n in (32, 40, 30, 30, 20)])
    with pytest.raises(RuntimeError, match="no cache pages"):
        t.U = t.W1.new_zeros((S.R, S.GAMMA, S.V))
        t.loop.round(t.U, t.logits)
    assert t.cache.held.tolist()[0] == 3
    # two requests end; the first one, 32 tokens on 2 pages and a reserved one, goes on twice
    t.cache.free(S.ints([1, 2]))
    assert t.cache.fork(S.ints([0]), S.ints([1])).tolist() == [0]
    t.kept[1], t.kept[2] = list(t.kept[0]), []
    assert t.cache.held.tolist()[:2] == [3, 2]
    for _ in range(2):
        t.round()
