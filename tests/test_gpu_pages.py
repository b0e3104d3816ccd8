"""Block tables and slot maps against the definition request by request: random
histories of batches, refusals when the blocks run out, padding, rows too short,
many tokens and many requests."""
import random

import pytest
import torch

import paged_ref as R

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


def up(a):
    return torch.tensor(a, dtype=I32, device="cuda")


class Both:
    """The same state on the host and on the GPU."""

    def __init__(self, K, rows, max_blocks, bs, free):
        self.K, self.bs = K, bs
        self.host = R.Pages(rows, max_blocks, bs, free)
        self.lens, self.held = up([0] * rows), up([0] * rows)
        self.table = torch.full((rows, max_blocks), -1, dtype=I32, device="cuda")
        self.free, self.count = up(free), up([len(free)])

    def tables(self):
        return self.lens, self.held, self.table, self.free, self.count

    def same(self):
        h = self.host
        assert self.lens.tolist() == h.lens and self.held.tolist() == h.held and self.count.tolist() == [h.count]
        assert self.table.tolist() == h.table and self.free.tolist()[:h.count] == h.free[:h.count]

    def reserve(self, lens, idx, extra=0):
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        T = cu[-1] + extra
        slots, totals = self.K.kv_reserve(up(cu), T, up(idx), *self.tables(), block_size=self.bs)
        want, sums = self.host.reserve(cu, idx, T)
        assert slots.tolist() == want and totals.tolist() == sums
        self.same()
        return cu, slots, totals

    def commit(self, cu, idx, steps=None):
        self.K.kv_commit(up(cu), up(idx), self.lens, self.held, block_size=self.bs, steps=None if steps is None else up(steps))
        self.host.commit(cu, idx, steps)
        self.same()

    def release(self, idx, keep=None):
        self.K.kv_release(up(idx), *self.tables(), block_size=self.bs, keep_lens=None if keep is None else up(keep))
        self.host.release(idx, keep)
        self.same()


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("seed", [1, 2])
def test_histories(K, bs, seed):
    """Prompts, steps, drafts of which some stand, cuts and ends, in random batches,
    until the blocks run out and after."""
    r = random.Random(seed * 100 + bs)
    rows = 12
    free = list(range(40))
    r.shuffle(free)
    b = Both(K, rows, 9, bs, free)
    for _ in range(12):
        n = r.randint(0, rows - 1)
        idx = r.sample(range(rows), n) + r.choice([[], [-1, -7], [rows]])
        lens = [r.choice([0, 1, 1, 4, bs - 1, bs, bs + 1, r.randint(1, 5 * bs)]) if i < n else r.choice([0, 2]) for i in range(len(idx))]
        cu, _, _ = b.reserve(lens, idx, r.choice([0, 5]))
        b.commit(cu, idx, r.choice([None, [r.randint(-2, x + 1) for x in lens]]))
        gone = r.sample(range(rows), r.randint(0, 4)) + [-1]
        b.release(gone, r.choice([None, [r.randint(-1, 3 * bs) for _ in gone]]))


def test_list_is_restored(K):
    """Giving back what a call took leaves the list as it was; asking twice takes
    nothing more."""
    free = list(range(100, 0, -1))
    b = Both(K, 6, 20, 16, free)
    idx = [3, 0, 5]
    cu, slots, totals = b.reserve([40, 100, 16], idx)
    again, sums = K.kv_reserve(up(cu), cu[-1], up(idx), *b.tables(), block_size=16)
    assert torch.equal(again, slots) and torch.equal(sums, totals)
    b.same()
    b.release(idx, [0, 0, 0])
    assert b.free.tolist() == free and b.count.tolist() == [100]


@pytest.mark.parametrize("n,lo,hi,bs", [(1, 20000, 20000, 16), (5, 3000, 9000, 64), (3000, 0, 3, 16), (2500, 0, 40, 32), (1024, 1, 1, 16), (1025, 1, 1, 128)])
def test_many(K, n, lo, hi, bs):
    """More tokens than one workgroup writes slots of, more requests than it has
    threads."""
    r = random.Random(n)
    lens = [r.randint(lo, hi) for _ in range(n)]
    most = max(-(-x // bs) for x in lens) + 1
    free = list(range(sum(-(-x // bs) for x in lens) - (3 if n > 2000 else 0)))   # the last do not get theirs
    r.shuffle(free)
    b = Both(K, n + 3, most, bs, free)
    idx = r.sample(range(n + 3), n)
    cu, _, _ = b.reserve(lens, idx)
    b.commit(cu, idx)
    b.reserve([1] * n, idx, 9)
    b.release(idx[::2])


def test_empty(K):
    b = Both(K, 3, 4, 16, [0, 1, 2])
    b.reserve([], [])
    b.reserve([], [], 4)
    b.reserve([0, 0], [1, -1])
    b.commit([0], [])
    b.release([])
    none = Both(K, 3, 4, 16, [])
    none.reserve([1, 0], [1, 2])
    none.release([1])


def test_full_list_and_odd_state(K):
    """A list without room drops what does not fit; negative counts and lengths of
    a state nobody filled count as none, and counts beyond the list as its length."""
    lens, held, table = up([0, 40]), up([0, 3]), up([[-1] * 4, [7, 8, 9, -1]])
    free, count = up([1, 2]), up([1])
    K.kv_release(up([1]), lens, held, table, free, count, block_size=16)
    assert free.tolist() == [1, 9] and count.tolist() == [2] and held.tolist() == [0, 0]
    for c, want in ((-5, []), (99, [2, 1])):
        lens, held, table, count = up([-3, 0]), up([-4, 0]), up([[-1] * 4, [-1] * 4]), up([c])
        slots, totals = K.kv_reserve(up([0, 17]), 17, up([0]), lens, held, table, up([1, 2]), count, block_size=16)
        assert totals.tolist() == [17 if want else 0] and table[0].tolist()[:2] == (want or [-1, -1])
        assert slots.tolist() == ([32 + i for i in range(16)] + [16] if want else [-1] * 17)
