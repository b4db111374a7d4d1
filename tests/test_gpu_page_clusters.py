"""Shared pages with every number of CTAs that the calls take: batches of 65 to 224
rows, wide tables and pools of 8 to 33 thousand pages."""
import numpy as np
import pytest

from oracle import shared as S
from test_gpu_shared_pages import Pool
from test_oracle_shared import state

pytestmark = pytest.mark.gpu

# rows, table columns behind the used ones, spare pages: 32 pieces of rows (of 256 columns) a CTA, or 4096 pages
CASES = [(b, 0, 300) for b in (33, 65, 96, 97, 130, 165, 200, 224, 225)] + [(40, 600, 60), (70, 300, 60)] + [(5, 0, n) for n in (8300, 12400, 16500, 20600, 24700, 28800)]


@pytest.mark.parametrize("B,extra,spare", CASES)
@pytest.mark.parametrize("chained", [False, True])
def test_steps_match_oracle(B, extra, spare, chained):
    P, r = 16, np.random.default_rng(B + spare + extra)
    lens = r.integers(0, 150, B)
    table, free, count, shares = state(B, P, lens, spare, B, extra + 2)
    pool = Pool(table, lens, shares, free, count, P)
    for turn in range(3):
        if chained:  # rows that change are read
            parents = r.integers(-1, B, B)
        else:        # only rows that stay are
            parents = np.where(r.random(B) < 0.5, np.arange(B), r.integers(0, (B + 3) // 4, B))
            parents[:(B + 3) // 4] = np.arange((B + 3) // 4)
        assert pool.fork(parents)["info"][0] == 0
        assert pool.own(r.integers(0, 2, B))["info"][0] in (0, S.NO_FREE)
        assert pool.release(np.where(r.random(B) < 0.6, -1, r.integers(0, 150, B)))["info"][0] == 0
        assert pool.compact()["info"][0] == 0


@pytest.mark.parametrize("B,extra,spare", CASES)
def test_refusals_change_nothing(B, extra, spare):
    P, r = 16, np.random.default_rng(B + 1)
    lens = r.integers(17, 150, B)
    table, free, count, shares = state(B, P, lens, spare, B, extra)
    fork = lambda t=table, s=shares, f=free, p=np.full(B, -1): Pool(t.copy(), lens, s.copy(), f.copy(), count, P).fork(p)["info"]  # noqa: E731
    bad = table.copy()
    bad[B - 1, 1] = len(shares)
    assert fork(t=bad) == [S.BAD_PAGE, 0]
    bad[B - 1, 1], bad[B // 2, 0] = bad[0, 0], bad[0, 0]  # two rows more than its shares say
    assert fork(t=bad) == [S.BAD_SHARES, 0]
    assert fork(f=free[:count + 1]) == [S.NO_FREE, 0]
    parents = np.arange(B)
    parents[B - 1] = B
    assert fork(p=parents) == [S.BAD_LENGTH, 0]
    moves = int((S.pages_compact(table, lens, shares, free, count, P, len(shares))["src"] >= 0).sum())
    if moves:
        assert Pool(table.copy(), lens, shares.copy(), free, count, P).compact(moves - 1)["info"] == [S.TOO_MANY_MOVES, 0]
    twice = free.copy()
    twice[count - 1] = twice[0]
    assert Pool(table.copy(), lens, shares.copy(), twice, count, P).compact()["info"] == [S.BAD_PAGE, 0]
