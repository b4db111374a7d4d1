"""A refusal within a step of shared pages, carried forward on the device: nothing
of the step is done, without the host looking at a call's info."""
import numpy as np
import pytest
import torch

from exact_attention_attn_gb300 import (attn_fwd_status, attn_kv8_append, attn_kv8_cache, attn_pages_assign, attn_pages_copy,
                                        attn_pages_fork, attn_pages_own)
from oracle import shared as S

pytestmark = pytest.mark.gpu

AFTER = 128


def _dev(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Step:
    """Rows that share page 0, some of it filled, and a stack of `free` pages; a step of one token a row."""

    def __init__(self, B=2, P=16, free=0, held=5):
        self.B, self.P = B, P
        pages = 1 + B
        self.table, self.lens = _dev([[0, -1]] * B), _dev([held] * B)
        self.shares, self.free, self.count = _dev([B - 1] + [0] * B), _dev(np.arange(1, pages)), _dev([free])
        self.new, self.parents = _dev([1] * B), _dev(np.arange(B))
        self.cache = attn_kv8_cache(pages, 1, 64, P)
        g = torch.Generator().manual_seed(1)
        self.k = torch.randn((B, 1, 64), generator=g).to(torch.bfloat16).cuda()
        old = torch.randn((held, 1, 64), generator=g).to(torch.bfloat16).cuda()
        attn_kv8_append(old, old, _dev(np.arange(held)), self.cache, P)
        self.info = [torch.empty(2, dtype=torch.int32, device="cuda") for _ in range(3)]
        self.slots, self.cu = _dev([7] * B), _dev([7] * (B + 1))

    def state(self):
        return [t.clone() for t in (self.table, self.lens, self.shares, self.free, self.count, self.cache)]

    def __call__(self, one_info=False):
        a, b, c = self.info[:1] * 3 if one_info else self.info
        counts = {"free_count": self.count}
        attn_pages_fork(self.table, self.lens, self.parents, self.shares, self.free, self.count, self.P,
                        out={**counts, "lens": self.lens, "info": a})
        own = attn_pages_own(self.table, self.lens, self.new, self.shares, self.free, self.count, self.P, out={**counts, "info": b}, after=a)
        attn_pages_copy(self.cache, own["src"], own["dst"])
        attn_pages_assign(self.table, self.lens, self.new, self.free, self.count, self.P, self.B, after=b,
                          out={**counts, "lens": self.lens, "slots": self.slots, "cu": self.cu, "info": c})
        attn_kv8_append(self.k, self.k, self.slots, self.cache, self.P)


@pytest.mark.parametrize("one_info", [False, True])
@pytest.mark.parametrize("B,P", [(2, 16), (2, 64), (9, 32), (300, 16), (3000, 16)])
def test_a_refused_own_leaves_the_step_undone(B, P, one_info):
    # as many free pages as rows that need one, less one
    s = Step(B, P, free=B - 2)
    before = s.state()
    s(one_info)
    assert all(torch.equal(x, y) for x, y in zip(before, s.state()))
    assert (s.slots == -1).all() and (s.cu == 0).all() and s.info[0 if one_info else 2].tolist() == [AFTER, 0]
    if not one_info:
        assert s.info[0].tolist() == [0, 0] and s.info[1].tolist() == [S.NO_FREE, 0]
    s.count += 1
    s(one_info)  # the same step with a page more
    assert s.info[0 if one_info else 2].tolist() == [0, B]
    assert len(set(s.slots.tolist())) == B and (s.slots % P == 5).all() and (s.lens == 6).all() and (s.shares == 0).all()
    assert not torch.equal(before[-1], s.cache) and attn_fwd_status() == 0


def test_a_refused_fork_leaves_the_step_undone():
    s = Step(4, 16, free=4)
    s.parents.copy_(_dev([0, 0, 4, 3]))  # no such row
    before = s.state()
    s()
    assert all(torch.equal(x, y) for x, y in zip(before, s.state()))
    assert (s.slots == -1).all() and [x.tolist() for x in s.info] == [[S.BAD_LENGTH, 0], [AFTER, 0], [AFTER, 0]]


def test_bits_of_the_own_call_are_told_as_well():
    s = Step(2, 16, free=2)
    s.info[0].copy_(_dev([S.BAD_PAGE, 3]))
    s.new.copy_(_dev([1, -1]))
    own = attn_pages_own(s.table, s.lens, s.new, s.shares, s.free, s.count, s.P, after=s.info[0])
    assert own["info"].tolist() == [AFTER | S.BAD_LENGTH, 0] and own["src"].tolist() == own["dst"].tolist() == [-1, -1]
    step = attn_pages_assign(s.table, s.lens, s.new, s.free, s.count, s.P, 1, after=own["info"])
    assert step["info"].tolist() == [AFTER | S.BAD_LENGTH, 0] and step["slots"].tolist() == [-1]
    assert step["lens"].tolist() == [5, 5] and step["free_count"].tolist() == [2]


def test_captured_steps_stop_and_go_on():
    s = Step(3, 16, free=2)
    s()  # (a first call outside of the capture; it is done)
    assert s.info[2].tolist() == [0, 3]
    s = Step(3, 16, free=1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s()
    before = s.state()
    for _ in range(3):
        g.replay()
        assert all(torch.equal(x, y) for x, y in zip(before, s.state())) and s.info[2].tolist() == [AFTER, 0]
    s.count += 1
    for turn in range(11):  # up to the end of the page, and a page more that the stack does not have
        g.replay()
        assert s.info[2].tolist() == [0, 3] and (s.lens == 6 + turn).all()
    g.replay()
    assert s.info[1].tolist() == [0, 0] and s.info[2].tolist() == [S.NO_FREE, 0] and (s.lens == 16).all()
    assert attn_fwd_status() == 0
