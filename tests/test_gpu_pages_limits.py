"""Block tables at the largest sizes that 32 bits describe: 2^31 - 1 slots, and 2^31 - 1
requests, all but a few of them padding."""
import pytest
import torch

pytestmark = pytest.mark.gpu
I32 = torch.int32
MOST = (1 << 31) - 1


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


def up(a):
    return torch.tensor(a, dtype=I32, device="cuda")


def test_most_slots(K):
    lens, held, table = up([0, 5, 0]), up([0, 1, 0]), up([[-1] * 4, [9, -1, -1, -1], [-1] * 4])
    free, count = up([3, 1, 7]), up([3])
    slots, totals = K.kv_reserve(up([0, 20, 40]), MOST, up([1, 0]), lens, held, table, free, count, block_size=16)
    assert totals.tolist() == [25, 20] and count.tolist() == [0] and held.tolist() == [2, 2, 0]
    want = [9 * 16 + 5 + i for i in range(11)] + [7 * 16 + i for i in range(9)] + [16 + i for i in range(16)] + [48 + i for i in range(4)]
    assert slots[:40].tolist() == want
    rest = slots[40:]
    for i in range(0, len(rest), 1 << 28):
        assert bool((rest[i:i + (1 << 28)] == -1).all()), i


def test_most_requests(K):
    cu = torch.zeros(MOST + 1, dtype=I32, device="cuda")
    idx = torch.full((MOST,), -1, dtype=I32, device="cuda")
    cu[1:] = 4
    cu[MOST] = 9                        # the last request has five tokens, the first four
    idx[0], idx[MOST - 1], idx[MOST // 2] = 2, 0, 1
    lens, held = up([10, 20, 30]), up([1, 2, 3])
    K.kv_commit(cu, idx, lens, held, block_size=16)
    assert lens.tolist() == [15, 20, 34]
