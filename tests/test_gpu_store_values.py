"""Every finite e4m3 number and every midpoint of two neighbours, both signs, stored
under a scale of one and others: the codes are known without arithmetic."""
import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF, I32, F8 = torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def K():
    import gated_delta_rule_51_amd as kda
    kda.lib()
    return kda


def every():
    """(values, codes) [rows, 64]: the first of a row is 448, which sets its scale."""
    codes = torch.arange(127)
    vals = codes.to(torch.uint8).view(F8).double()
    mids = (vals[1:] + vals[:-1]) / 2
    even = codes[:-1] + codes[:-1] % 2                    # of two neighbours the even one
    x, c = torch.cat([vals, mids, -vals, -mids]), torch.cat([codes, even, codes + 128, even + 128])
    more = -len(x) % 63
    x, c = torch.cat([x, torch.zeros(more, dtype=x.dtype)]), torch.cat([c, torch.zeros(more, dtype=c.dtype)])
    x = torch.cat([torch.full((len(x) // 63, 1), 448.0, dtype=x.dtype), x.view(-1, 63)], 1)
    c = torch.cat([torch.full((len(c) // 63, 1), 0x7e), c.view(-1, 63)], 1)
    return x, c.to(torch.uint8)


def test_list_is_whole():
    x, c = every()
    finite = [i for i in range(256) if i & 0x7f != 0x7f]
    assert sorted(set(c.flatten().tolist())) == finite
    vals = torch.arange(127, dtype=torch.uint8).view(F8).double()
    for sign in (1, -1):
        given = set((sign * x[:, 1:]).flatten().tolist())
        assert all(v in given for v in vals.tolist())
        assert all(m in given for m in ((vals[1:] + vals[:-1]) / 2).tolist())


@pytest.mark.parametrize("io", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("exponent", [0, -20, 17])
@pytest.mark.parametrize("run", [1, 3, 9], ids=["single", "short", "long"])
def test_codes(K, io, exponent, run):
    """Each row in a block of its own, and in runs that a wave or a workgroup stores."""
    x, c = every()
    n, bs = len(x), 16
    assert n == 9 and torch.equal(x.to(BF).double(), x)
    x = (x * 2.0 ** exponent).to(io)
    kc = torch.full((n, 1, bs, 64), 0x55, dtype=torch.uint8, device="cuda")
    vc = torch.full((n, 1, 64, bs), 0x55, dtype=torch.uint8, device="cuda")
    ks, vs = (torch.full((n, 1), float("nan"), device="cuda") for _ in range(2))
    slots = [i // run * bs + i % run for i in range(n)]
    K.kv_store(x.view(n, 1, 64).cuda(), (-x).view(n, 1, 64).cuda(), torch.tensor(slots, dtype=I32, device="cuda"), kc.view(F8), vc.view(F8), ks, vs)
    want = torch.full((n, bs, 64), 0x55, dtype=torch.uint8)
    minus = want.clone()
    for i in range(n):
        want[slots[i] // bs, slots[i] % bs] = c[i]
        minus[slots[i] // bs, slots[i] % bs] = c[i] ^ 0x80
    assert torch.equal(kc.cpu()[:, 0], want)
    assert torch.equal(vc.cpu()[:, 0].transpose(1, 2), minus)
    used = -(-n // run)
    assert ks.tolist()[:used] == [[2.0 ** exponent]] * used and vs.tolist()[:used] == [[2.0 ** exponent]] * used
    assert bool(ks[used:].isnan().all())
