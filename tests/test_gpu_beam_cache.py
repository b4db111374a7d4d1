"""A beam search over the 8-bit cache: the device's cache is the oracle's, bit for bit,
after every step, fork, compaction and release."""
import numpy as np
import pytest

from test_gpu_beam import Search
from test_gpu_kv8 import _check_cache

pytestmark = pytest.mark.gpu


class Checked(Search):
    def same(self):
        """Codes, scales and marks of every block that was ever begun, and each row's tokens."""
        _check_cache(self.model, self.cache, self.D, self.P)
        table, lens = self.table.cpu().numpy(), self.lens.cpu().numpy()
        for side in range(2):
            value = self.model.values(side)
            for r in range(self.B):
                pos = np.arange(lens[r])
                slots = table[r, pos // self.P] * self.P + pos % self.P
                told = np.array([t[side] for t in self.told[r]]).reshape(len(slots), self.H, self.D)
                unit = np.array([2.0 ** self.model.exp[side][s // 16].astype(float) for s in slots]).reshape(len(slots), self.H, 1)
                # One rounding when written (2^-4 relative, or 2^-10 of the block's unit), and where the unit grows by 2^d
                # codes are exact but for e4m3's smallest numbers: 2^-10 of the new unit.  Units at least double, so
                # those sum to 2^-9 of the last one.
                assert (np.abs(value[slots] - told) <= 2.0 ** -4 * np.abs(told) + 2.0 ** -9 * unit).all(), r

    def fork(self, parents):
        super().fork(parents)
        self.same()

    def compact(self):
        super().compact()
        self.same()

    def release(self, keep):
        super().release(keep)
        self.same()

    def step(self, new, seed):
        super().step(new, seed)
        self.same()


@pytest.mark.parametrize("B,H,Hq,D,P", [(6, 2, 8, 64, 16), (8, 1, 4, 128, 32), (5, 2, 2, 192, 64), (7, 1, 2, 256, 16)])
def test_the_cache_through_a_beam_search(B, H, Hq, D, P):
    r = np.random.default_rng(B + D)
    s = Checked(B, H, Hq, D, P, pages=B * 8, width=7)
    s.step([int(n) if b % 2 == 0 else 0 for b, n in enumerate(r.integers(1, 3 * P, B))], 1)
    s.fork([b - b % 2 for b in range(B)])
    for turn in range(8):
        s.step(r.integers(0, 4, B), 10 * turn + 20)
        s.fork([int(p) if r.random() < 0.4 else b for b, p in enumerate(r.integers(0, B, B))])
        if turn % 2:
            s.release([int(r.integers(max(0, n - 20), n + 1)) if r.random() < 0.5 else -1 for n in s.lens.tolist()])  # often inside a block
        if turn % 3 == 1:
            s.compact()
    s.release([0] * B)
    assert int(s.count) == s.pages
