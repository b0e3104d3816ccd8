"""Requests that did not get their blocks: nothing of theirs is counted, whichever
step of their run would have stood, and the tables stay as the definition says."""
import random

import pytest
import torch

import paged_ref as R
from test_gpu_pages import Both, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


class Pages(R.Pages):
    def commit(self, cu, idx, steps=None):
        """Only the tokens of a run that has blocks for all of itself were stored."""
        for n, r in enumerate(idx):
            L = cu[n + 1] - cu[n]
            s = L - 1 if steps is None else steps[n]
            if 0 <= r < len(self.lens) and 0 <= s < L and self.lens[r] + L <= self.held[r] * self.bs:
                self.lens[r] += s + 1


class Same(Both):
    def __init__(self, K, rows, max_blocks, bs, free):
        super().__init__(K, rows, max_blocks, bs, free)
        self.host = Pages(rows, max_blocks, bs, free)


def test_refused_drafts_do_not_count(K):
    """14 tokens in the only block, four drafts of which two are said to stand: none
    was stored, so the length stays, with and without steps; what fits counts."""
    b = Same(K, 3, 4, 16, [5])
    cu, _, _ = b.reserve([14], [1])
    b.commit(cu, [1])
    for steps in ([0], [1], [3], None):
        cu, slots, totals = b.reserve([4], [1])
        assert slots.tolist() == [-1] * 4 and totals.tolist() == [0]
        b.commit(cu, [1], steps)
        assert b.lens.tolist() == [0, 14, 0]
    cu, _, totals = b.reserve([2], [1])
    assert totals.tolist() == [16]
    b.commit(cu, [1], [0])
    assert b.lens.tolist() == [0, 15, 0]


def test_row_too_short(K):
    """A run beyond the row's entries is refused and not counted either."""
    b = Same(K, 2, 2, 16, list(range(8)))
    cu, _, _ = b.reserve([30], [0])
    b.commit(cu, [0])
    cu, _, totals = b.reserve([4], [0])
    assert totals.tolist() == [0]
    b.commit(cu, [0], [1])
    assert b.lens.tolist() == [30, 0]


@pytest.mark.parametrize("steps,want", [(None, 17), ([4], 5)])
def test_length_nobody_filled(K, steps, want):
    """A negative length counts as none for the reservation, and so for what follows."""
    lens, held, table = up([-3]), up([0]), up([[-1, -1]])
    free, count = up([4, 2]), up([2])
    slots, totals = K.kv_reserve(up([0, 17]), 17, up([0]), lens, held, table, free, count, block_size=16)
    assert totals.tolist() == [17] and slots.tolist() == [32 + i for i in range(16)] + [64]
    K.kv_commit(up([0, 17]), up([0]), lens, held, block_size=16, steps=None if steps is None else up(steps))
    assert lens.tolist() == [want]


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("seed", [3, 4, 5])
def test_histories(K, bs, seed):
    """Few blocks and many runs: most histories refuse some with room left for a part
    of them; totals of 0 and lengths that stay go together."""
    r = random.Random(seed * 1000 + bs)
    rows = 9
    b = Same(K, rows, 6, bs, r.sample(range(100), 14))
    refused = 0
    for _ in range(25):
        idx = r.sample(range(rows), r.randint(1, rows)) + r.choice([[], [-1]])
        lens = [r.choice([1, 2, 4, bs // 2, bs, r.randint(1, 2 * bs)]) for _ in idx]
        cu, _, totals = b.reserve(lens, idx)
        before, totals = b.lens.tolist(), totals.tolist()
        b.commit(cu, idx, r.choice([None, [r.randint(-1, x) for x in lens], [0] * len(idx)]))
        for i, n in zip(idx, totals):
            if 0 <= i < rows and n == 0:
                refused += 1
                assert b.lens.tolist()[i] == before[i]
        if r.random() < 0.5:
            gone = r.sample(range(rows), r.randint(1, 3))
            b.release(gone, r.choice([None, [bs // 2] * len(gone)]))
    assert refused > 3
    print("refused:", refused, flush=True)
