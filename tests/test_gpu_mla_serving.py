"""GPU tests of the paged cache of the full-context (MLA) layers in a server's use, and of what its inputs may get wrong."""
import pytest
import torch
from test_gpu_mla_paged import D, Cache, hd, i32  # noqa: F401  (hd: a fixture)

pytestmark = pytest.mark.gpu


def bits(t):
    return t.view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(a, b):
    return torch.equal(bits(a.contiguous()), bits(b.contiguous()))


def places(c, b, rows):
    i = torch.tensor(rows, device="cuda")
    return c.table[b].long()[i // c.page], i % c.page


def expect_bounds_error(hd):  # noqa: F811
    with pytest.raises(hd.HcaDsaError, match="DEVICE_BOUNDS"):
        hd.hcadsa_check_device_error()


# ----------------------------------------------------------------------------- lengths out of range


@pytest.mark.parametrize("kv0", [33, 34, 36, 37, 1 << 30, 2 ** 31 - 1, 3, 0, -5, -(2 ** 31)])
def test_append_outside_the_table(hd, kv0):  # noqa: F811
    """Four new rows of a sequence whose length does not fit its table row (32 rows): those that have a place are
    written there, the others nowhere, and the sequence's other rows keep theirs."""
    c = Cache([4, 2], [32, 20], Hq=4, page=16, seed=7)
    k, v = c.rand(6, 1, D), c.rand(6, 1, D)
    pos = torch.full(c.K.shape[:3], -5, dtype=i32, device="cuda")
    mass = torch.full(c.K.shape[:3], 3.0, device="cuda")
    want = [x.clone() for x in (c.K, c.V, pos, mass)]
    seen = torch.tensor([1000, 20], dtype=i32, device="cuda")
    for b, end, t0, n in ((0, kv0, 0, 4), (1, 20, 4, 2)):
        for i in range(n):
            r = end - n + i
            if 0 <= r < 32:
                at = places(c, b, [r])
                want[0][at], want[1][at] = k[t0 + i], v[t0 + i]
                want[2][at], want[3][at] = (1000 if b == 0 else 20) - n + i, 0.0
    kv = torch.tensor([kv0, 20], dtype=i32, device="cuda")
    hd.mla_cache_append(k, v, c.K, c.V, c.table, c.cu, kv, seen=seen, pos=pos, mass=mass)
    expect_bounds_error(hd)
    for got, ref in zip((c.K, c.V, pos, mass), want):
        assert same(got, ref)


def test_append_of_a_cut_batch(hd):  # noqa: F811
    """cu_q reaches beyond the packed rows: the rows that are there go where they belong."""
    c = Cache([4, 8], [20, 40], Hq=4, page=16, seed=8)
    k, v = c.rand(9, 1, D), c.rand(9, 1, D)  # five of the second sequence's eight
    pos = torch.full(c.K.shape[:3], -5, dtype=i32, device="cuda")
    want = [x.clone() for x in (c.K, c.V, pos)]
    for b, r0, t0, n in ((0, 16, 0, 4), (1, 32, 4, 5)):
        at = places(c, b, list(range(r0, r0 + n)))
        want[0][at], want[1][at] = k[t0 : t0 + n], v[t0 : t0 + n]
        want[2][at] = torch.arange(r0, r0 + n, dtype=i32, device="cuda")[:, None]
    hd.mla_cache_append(k, v, c.K, c.V, c.table, c.cu, c.kv_len, pos=pos)
    expect_bounds_error(hd)
    for got, ref in zip((c.K, c.V, pos), want):
        assert same(got, ref)
