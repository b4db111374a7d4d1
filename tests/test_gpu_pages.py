"""Pages handed out and taken back on the GPU, bit for bit against the oracle."""
import numpy as np
import pytest
import torch

from exact_attention_attn_gb300 import attn_pages_assign, attn_pages_release
from oracle import serving as S

pytestmark = pytest.mark.gpu


def _dev(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _state(B, P, width, lens, spare, seed):
    """A table whose requests hold their pages, and a shuffled stack of the others."""
    r = np.random.default_rng(seed)
    have = -(-np.asarray(lens) // P)
    ids = r.permutation(int(have.sum()) + spare)
    table, at = np.full((B, width), -1), 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    free = np.concatenate([ids[at:], np.full(at, -9)])
    return table, free, spare


def _same(got, want, table, names):
    assert np.array_equal(table.cpu().numpy(), want["table"])
    assert got["info"].tolist() == want["info"]
    for n in names:
        assert np.array_equal(got[n].cpu().numpy(), np.atleast_1d(want[n])), n


CASES = [
    # B, P, longest cached, longest new, table slack, spare pages, padding
    (1, 16, 0, 1, 0, 4, 0),
    (1, 16, 15, 1, 0, 4, 3),
    (1, 64, 64, 1, 2, 1, 2),
    (7, 32, 100, 40, 1, 60, 5),
    (600, 16, 300, 1, 0, 700, 9),
    (513, 64, 0, 90, 3, 1500, 1),
    (5000, 32, 40, 3, 1, 9000, 0),
    (3, 16, 2000, 9000, 2, 3000, 100),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("inplace", [False, True])
def test_assign_and_release(case, inplace):
    B, P, lmax, nmax, slack, spare, pad = case
    r = np.random.default_rng(B + P)
    lens = r.integers(0, lmax + 1, B)
    new = r.integers(0, nmax + 1, B)
    new[r.integers(0, B)] = nmax
    width = int(-(-(lens + new).max() // P)) + slack
    table, free, count = _state(B, P, width, lens, spare, seed=B)
    most = int(new.sum()) + pad
    want = S.pages_assign(table, lens, new, free, count, P, most)
    assert want["info"][0] == 0
    dt, dl, df, dc = _dev(table), _dev(lens), _dev(free), _dev([count])
    out = {"lens": dl, "free_count": dc} if inplace else None
    got = attn_pages_assign(dt, dl, _dev(new), df, dc, P, most, out=out)
    _same(got, want, dt, ("lens", "free_count", "cu", "slots", "positions"))
    assert np.array_equal(df.cpu().numpy(), free)
    if not inplace:
        assert np.array_equal(dl.cpu().numpy(), lens) and dc.item() == count
    # then cut some requests, finish some, leave some
    keep = np.where(r.random(B) < 0.3, -1, r.integers(0, want["lens"].max() + 2, B))
    keep[r.random(B) < 0.2] = 0
    back = S.pages_release(want["table"], want["lens"], keep, free, want["free_count"], P)
    assert back["info"][0] == 0
    state = {"lens": got["lens"], "free_count": got["free_count"]}
    rel = attn_pages_release(dt, got["lens"], _dev(keep), df, got["free_count"], P, out=state if inplace else None)
    _same(rel, back, dt, ("lens", "free_count"))
    assert np.array_equal(df.cpu().numpy(), back["free"])


@pytest.mark.parametrize("what", ["length", "negative", "tokens", "pages", "count", "count_negative", "huge"])
def test_refused_steps_change_nothing(what):
    B, P = 40, 16
    lens = np.arange(B) * 3
    new = np.full(B, 5)
    table, free, count = _state(B, P, 10, lens, 30, seed=1)
    most = 5 * B
    if what == "length":
        new[7] = 10 * P - lens[7] + 1
        most = 10000
    elif what == "negative":
        lens = lens.copy()
        lens[3] = -1
    elif what == "tokens":
        most -= 1
    elif what == "pages":
        count = 3
    elif what == "count":
        count = len(free) + 1
    elif what == "count_negative":
        count = -1
    else:  # sums past 32 bits
        new[:] = 2 ** 31 - 1
    want = S.pages_assign(table, lens, new, free, count, P, most)
    assert want["info"][0] != 0
    dt, df = _dev(table), _dev(free)
    got = attn_pages_assign(dt, _dev(lens), _dev(new), df, _dev([count]), P, most)
    _same(got, want, dt, ("lens", "free_count", "cu", "slots", "positions"))
    assert np.array_equal(df.cpu().numpy(), free)


def test_refused_release():
    lens = np.array([40, 70])
    table, free, count = _state(2, 16, 6, lens, 3, seed=2)
    for free_, lens_, count_ in ((free[:5], lens, 3), (free, np.array([40, 97]), 3), (free, lens, -2), (free, lens, 99)):
        want = S.pages_release(table, lens_, [0, 0], free_, count_, 16)
        assert want["info"][0] != 0
        dt, df = _dev(table), _dev(free_)
        got = attn_pages_release(dt, _dev(lens_), _dev([0, 0]), df, _dev([count_]), 16)
        _same(got, want, dt, ("lens", "free_count"))
        assert np.array_equal(df.cpu().numpy(), free_)


def test_empty_and_strided_table():
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    got = attn_pages_assign(z.reshape(0, 4), z, z, _dev([1, 2]), _dev([2]), 16, 3)
    assert got["cu"].tolist() == [0] and got["slots"].tolist() == [-1] * 3 and got["free_count"].item() == 2
    assert attn_pages_release(z.reshape(0, 4), z, z, _dev([1, 2]), _dev([2]), 16)["info"].tolist() == [0, 0]
    wide = _dev(np.full((3, 9), -5))
    got = attn_pages_assign(wide[:, :4], _dev([0, 0, 0]), _dev([17, 0, 64]), _dev(np.arange(9)), _dev([9]), 16, 81)
    assert got["info"].tolist() == [0, 81]
    assert wide.tolist() == [[8, 7, -5, -5] + [-5] * 5, [-5] * 9, [6, 5, 4, 3] + [-5] * 5]


@pytest.mark.parametrize("P", [16, 64])
def test_pages_without_a_slot(P):
    # ids whose slots 32 bits do not hold, and ids below 0, on the stack and in the table
    top = 2 ** 31 // P
    table = np.array([[5, top, -1, -1, -1], [-1, -1, -1, -1, -1], [-7, -1, -1, -1, -1]])
    free = np.array([3, -2 ** 31, top - 1, top, -1, 2 ** 31 - 1])
    lens, new = np.array([P + 3, 0, 2]), np.array([2 * P, 3 * P, 5])
    want = S.pages_assign(table, lens, new, free, 6, P, 6 * P)
    assert want["info"][0] == 0 and set(want["slots"][want["slots"] < 0]) == {-2, -1}
    dt = _dev(table)
    got = attn_pages_assign(dt, _dev(lens), _dev(new), _dev(free), _dev([6]), P, 6 * P)
    _same(got, want, dt, ("lens", "free_count", "cu", "slots", "positions"))


def test_largest_batch():
    B, P = 16384, 16
    lens = np.zeros(B, dtype=np.int64)
    new = np.arange(B) % 7
    free = np.arange(B)[::-1].copy()
    table = np.full((B, 1), -1)
    want = S.pages_assign(table, lens, new, free, B, P, int(new.sum()))
    dt = _dev(table)
    got = attn_pages_assign(dt, _dev(lens), _dev(new), _dev(free), _dev([B]), P, int(new.sum()))
    _same(got, want, dt, ("lens", "free_count", "cu", "slots", "positions"))


def test_assign_and_release_captured():
    # a captured step replayed on changed lengths, in place; and a release captured behind it
    B, P, width, cap = 9, 16, 12, 90
    table, lens, new, keep = _dev(np.full((B, width), -1)), _dev(np.zeros(B)), _dev(np.zeros(B)), _dev(np.full(B, -1))
    free, count = _dev(np.arange(cap)), _dev([cap])
    out = {"lens": lens, "free_count": count}
    out = attn_pages_assign(table, lens, new, free, count, P, 100, out=out)
    rel = attn_pages_release(table, lens, keep, free, count, P, out={"lens": lens, "free_count": count})
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn_pages_assign(table, lens, new, free, count, P, 100, out=out)
        attn_pages_release(table, lens, keep, free, count, P, out=rel)
    o_table, o_lens, o_free, o_count = np.full((B, width), -1), np.zeros(B, dtype=np.int64), np.arange(cap), cap
    r = np.random.default_rng(5)
    for _ in range(6):
        n, kp = r.integers(0, 12, B), np.where(r.random(B) < 0.7, -1, r.integers(0, 20, B))
        new.copy_(_dev(n))
        keep.copy_(_dev(kp))
        g.replay()
        a = S.pages_assign(o_table, o_lens, n, o_free, o_count, P, 100)
        assert a["info"][0] == 0
        b = S.pages_release(a["table"], a["lens"], kp, o_free, a["free_count"], P)
        o_table, o_lens, o_free, o_count = b["table"], b["lens"], b["free"], b["free_count"]
        assert np.array_equal(out["slots"].cpu().numpy(), a["slots"]) and out["info"].tolist() == a["info"]
        assert np.array_equal(table.cpu().numpy(), o_table) and np.array_equal(lens.cpu().numpy(), o_lens)
        assert np.array_equal(free.cpu().numpy(), o_free) and count.item() == o_count and rel["info"].tolist() == b["info"]


@pytest.mark.parametrize("active", [[0, 4999], [4998, 4999], [0, 1, 2500, 2501, 4000], [7], [3, 1000, 1001, 1002, 4999], []])
def test_few_active_requests_among_idle_ones(active):
    # one to six tokens each, so that a thread's four tokens lie in requests far apart
    B, P = 5000, 16
    r = np.random.default_rng(len(active))
    lens, new = r.integers(0, 40, B), np.zeros(B, dtype=np.int64)
    new[active] = r.integers(1, 7, len(active))
    table, free, count = _state(B, P, 4, lens, 50, seed=3)
    most = int(new.sum()) + 3
    want = S.pages_assign(table, lens, new, free, count, P, most)
    dt = _dev(table)
    got = attn_pages_assign(dt, _dev(lens), _dev(new), _dev(free), _dev([count]), P, most)
    _same(got, want, dt, ("lens", "free_count", "cu", "slots", "positions"))


def test_idle_requests_cost_no_walk():
    # two active requests at the two ends of the largest batch take about the time of two that are neighbours
    B, P = 16384, 16
    times = []
    for active in ([0, 1], [0, B - 1]):
        new = np.zeros(B, dtype=np.int64)
        new[active] = 2
        args = (_dev(np.full((B, 1), -1)), _dev(np.zeros(B)), _dev(new), _dev(np.arange(8)), _dev([8]), P, 4)
        out = attn_pages_assign(*args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(10):
                attn_pages_assign(*args, out=out)
        best = float("inf")
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            g.replay()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
        assert out["slots"].tolist() == [7 * P, 7 * P + 1, 6 * P, 6 * P + 1]
    assert times[1] <= 2 * times[0], times
