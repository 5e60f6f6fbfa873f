"""GPU tests of the paged cache of the full-context (MLA) layers in a server's use, and of what its inputs may get wrong."""
import math

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


# ----------------------------------------------------------------------------- values that are not finite

FINITE = {
    "one_tile": dict(q_len=[1], kv_len=[40]),
    "few_pieces": dict(q_len=[1, 1], kv_len=[40, 300]),
    "many_pieces": dict(q_len=[1], kv_len=[40000]),
    "prompt": dict(q_len=[300], kv_len=[300], page=16),
    "whole_row_tiles": dict(q_len=[256], kv_len=[1024]),
    "chunk_pieces": dict(q_len=[70, 1], kv_len=[5000, 900], Hq=16, Hkv=2, page=32),
}


@pytest.mark.parametrize("where", ["Q", "K"])
@pytest.mark.parametrize("name", list(FINITE))
def test_nan_stays_visible(hd, name, where):  # noqa: F811
    """A NaN in a query, or in a cached row that a token sees, is a NaN in that token's O, lse and weights, whether
    or not its row tile was cut into pieces; nothing else changes."""
    c = Cache(seed=3, **FINITE[name])
    T, grp = c.q.shape[0], c.Hq // c.Hkv
    O, lse = hd.mla_paged_attn_fwd(c.q, *c.args(), return_lse=True)
    mass = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse)
    bad = torch.zeros((T, c.Hq), dtype=torch.bool, device="cuda")
    bad_row = torch.zeros(mass.shape, dtype=torch.bool, device="cuda")
    t0 = 0
    for b, n in enumerate(c.q_len):
        if where == "Q":
            for i, h in ((n - 1, 0), (n // 2, c.Hq - 1)):
                c.q[t0 + i, h, 5] = math.nan
                bad[t0 + i, h] = True
                at = places(c, b, list(range(c.kv[b] - n + i + 1)))
                bad_row[at[0], at[1], h // grp] = True
        else:
            row, kvh = c.kv[b] - (n + 1) // 2, c.Hkv - 1  # the last half of the tokens see it
            c.K[places(c, b, [row])[0], row % c.page, kvh, 200] = math.nan
            first = row - (c.kv[b] - n)
            bad[t0 + first : t0 + n, kvh * grp :] = True
            bad_row[c.rows(b)[0], c.rows(b)[1], kvh] = True
        t0 += n
    O2, lse2 = hd.mla_paged_attn_fwd(c.q, *c.args(), return_lse=True)
    mass2 = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse2)
    hd.hcadsa_check_device_error()
    assert torch.isnan(O2[bad]).all() and torch.isnan(lse2[bad]).all()
    assert same(O2[~bad], O[~bad]) and same(lse2[~bad], lse[~bad])
    assert torch.isnan(mass2[bad_row]).all() and same(mass2[~bad_row], mass[~bad_row])


# ----------------------------------------------------------------------------- scratch


@pytest.mark.parametrize("fill", [0xff, 0x01, 0x00])
def test_what_a_workspace_held_does_not_matter(hd, fill):  # noqa: F811
    """Small batches leave most workers without work: their records have to be written too."""
    for q_len, kv_len in (([1], [1]), ([1, 1], [300, 40]), ([70], [700]), ([0, 0], [5, 9])):
        c = Cache(q_len, kv_len, Hq=16, seed=19)
        T = max(1, sum(q_len))
        if not sum(q_len):
            c.q = c.rand(1, 16, D)
        O, lse = hd.mla_paged_attn_fwd(c.q, *c.args(), O=torch.ones_like(c.q), lse=torch.ones(T, 16, device="cuda"),
                                       return_lse=True)
        mass = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse)
        ws = [torch.full((getattr(hd.lib(), f + "_workspace_size")(len(q_len), T, 16, 1),), fill, dtype=torch.uint8,
                         device="cuda") for f in ("mla_paged_attn_fwd", "mla_paged_attn_mass")]
        O2, lse2 = hd.mla_paged_attn_fwd(c.q, *c.args(), O=torch.ones_like(c.q), lse=torch.ones(T, 16, device="cuda"),
                                         return_lse=True, workspace=ws[0])
        mass2 = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse, workspace=ws[1])
        hd.hcadsa_check_device_error()
        assert same(O2, O) and same(lse2, lse) and same(mass2, mass)
