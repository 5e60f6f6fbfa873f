"""GPU tests of the paged cache of the full-context (MLA) layers in a server's use, and of what its inputs may get wrong."""
import math
import os
import subprocess
import sys

import pytest
import torch
from test_gpu_mla_paged import CASES, D, Cache, bf, hd, i32, oracle  # noqa: F401  (hd: a fixture)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


def test_good_sequences_next_to_bad_ones(hd):  # noqa: F811
    """Pages that are not there in the second of three sequences: the other two get what they get alone."""
    c = Cache([4, 3, 2], [200, 150, 90], seed=11, Hq=16)
    table = c.table.clone()
    table[1, 0], table[1, 1], table[1, 2] = -1, 1 << 29, c.K.shape[0]
    good = [0, 2]
    O, lse = hd.mla_paged_attn_fwd(c.q, *c.args(), return_lse=True)
    mass = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse)
    pos = torch.zeros(c.K.shape[:3], dtype=i32, device="cuda")
    for b in range(3):
        pos[c.rows(b)] = torch.arange(c.kv[b], dtype=i32, device="cuda")[:, None]
    moves, new = hd.mla_evict_select(mass, pos, c.table, c.kv_len, None, 64, n_sink=2, n_recent=9)
    hd.hcadsa_check_device_error()

    O2, lse2 = hd.mla_paged_attn_fwd(c.q, c.K, c.V, table, c.cu, c.kv_len, return_lse=True)
    expect_bounds_error(hd)
    mass2 = hd.mla_paged_attn_mass(c.q, c.K, table, c.cu, c.kv_len, lse)
    expect_bounds_error(hd)
    moves2, new2 = hd.mla_evict_select(mass, pos, table, c.kv_len, None, 64, n_sink=2, n_recent=9)
    expect_bounds_error(hd)
    assert torch.equal(new2, new)
    for b, t in zip(good, (slice(0, 4), slice(7, 9))):
        assert same(O2[t], O[t]) and same(lse2[t], lse[t])
        assert same(mass2[c.rows(b)], mass[c.rows(b)])
        assert torch.equal(moves2[b], moves[b])
    rest = torch.ones(c.K.shape[0], dtype=torch.bool, device="cuda")
    rest[c.table[good].long()] = False
    assert (mass2[rest] == 0).all()

    new_k, new_v = c.rand(9, 1, D), c.rand(9, 1, D)
    for call in ("append", "move"):
        want, got = ([x.clone() for x in (c.K, c.V, pos, mass)] for _ in range(2))
        for state, tab in ((want, c.table), (got, table)):
            Kp, Vp, ps, ms = state
            if call == "append":
                hd.mla_cache_append(new_k, new_v, Kp, Vp, tab, c.cu, c.kv_len, pos=ps, mass=ms)
            else:
                hd.mla_cache_move(moves, Kp, Vp, tab, pos=ps, mass=ms)
            if tab is table:
                expect_bounds_error(hd)
            hd.hcadsa_check_device_error()
        for w, g, first in zip(want, got, (c.K, c.V, pos, mass)):
            for b in good:
                assert same(g[c.rows(b)], w[c.rows(b)])
            assert same(g[rest], first[rest])


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


# ----------------------------------------------------------------------------- the calls' own totals


@pytest.mark.parametrize("name", ["one_token_one_row", "decode_ragged", "decode_gqa", "long_chunk", "mixed",
                                  "chunk_gqa_fused_pool", "rows_that_see_nothing", "many_prompts", "long_decode"])
def test_weights_add_up(hd, name):  # noqa: F811
    """The weights of a K/V head add up to the number of (token, query head) rows that see anything: within the sum of
    the rows' own bounds, and of lse's (d + 2^-18 + 2^-22 |lse| + rows 2^-24, as a factor)."""
    c = Cache(seed=len(name), **CASES[name])
    O, lse = hd.mla_paged_attn_fwd(c.q, *c.args(), return_lse=True)
    mass = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse).double()
    hd.hcadsa_check_device_error()
    _, _, l64, d, _, tol = oracle(c, lse_in=lse)
    sees = l64 > -math.inf
    off = torch.where(sees, d + 2.0 ** -18 + 2.0 ** -22 * l64.abs() + max(c.kv) * 2.0 ** -24, 0.0)
    grp = c.Hq // c.Hkv
    for h in range(c.Hkv):
        rows = sees[:, h * grp : (h + 1) * grp]
        bound = tol[..., h].sum() + 1.01 * off[:, h * grp : (h + 1) * grp].sum()
        assert (mass[..., h].sum() - rows.sum()).abs() <= bound, (name, h)


# ----------------------------------------------------------------------------- streams, graphs, scratch


class Server:
    """The state of a server: pools, positions, weights, table and lengths, and the inputs of one step."""

    B, Hq, Hkv, page, width, T, budget, sink, recent = 5, 16, 2, 16, 24, 260, 96, 2, 20

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n_pages = self.B * self.width
        self.K, self.V = torch.full((2, n_pages, self.page, self.Hkv, D), math.nan, dtype=bf, device="cuda").unbind(0)
        self.pos = torch.zeros((n_pages, self.page, self.Hkv), dtype=i32, device="cuda")
        self.mass = torch.zeros((n_pages, self.page, self.Hkv), device="cuda")
        self.table = torch.randperm(n_pages, generator=g, device="cuda").reshape(self.B, self.width).to(i32)
        self.kv, self.seen = (torch.zeros(self.B, dtype=i32, device="cuda") for _ in range(2))
        self.cu = torch.zeros(self.B + 1, dtype=i32, device="cuda")
        self.q = torch.zeros((self.T, self.Hq, D), dtype=bf, device="cuda")
        self.k, self.v = (torch.zeros((self.T, self.Hkv, D), dtype=bf, device="cuda") for _ in range(2))
        self.O = torch.zeros_like(self.q)
        self.lse = torch.zeros((self.T, self.Hq), device="cuda")

    def take(self, n, seed):
        """New inputs, the same for every server that is given the same seed."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        for x in (self.q, self.k, self.v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        add = torch.tensor(n, dtype=i32, device="cuda")
        self.cu[1:] = add.cumsum(0)
        self.kv += add
        self.seen += add

    def step(self, hd, stream=None):  # noqa: F811
        hd.mla_cache_append(self.k, self.v, self.K, self.V, self.table, self.cu, self.kv, seen=self.seen, pos=self.pos,
                            mass=self.mass, stream=stream)
        hd.mla_paged_attn_fwd(self.q, self.K, self.V, self.table, self.cu, self.kv, O=self.O, lse=self.lse, stream=stream)
        hd.mla_paged_attn_mass(self.q, self.K, self.table, self.cu, self.kv, self.lse, mass=self.mass, stream=stream)
        self.moves, self.new = hd.mla_evict_select(self.mass, self.pos, self.table, self.kv, self.seen, self.budget,
                                                   n_sink=self.sink, n_recent=self.recent, stream=stream)
        hd.mla_cache_move(self.moves, self.K, self.V, self.table, pos=self.pos, mass=self.mass, stream=stream)

    def state(self):
        return self.K, self.V, self.pos, self.mass, self.O, self.lse, self.moves, self.kv


STEPS = [[100, 0, 3, 90, 1], [1, 1, 1, 1, 1], [40, 120, 0, 33, 7], [0, 0, 0, 0, 0], [1, 0, 200, 1, 1], [1, 1, 1, 1, 1],
         [52, 52, 52, 52, 52]]


def test_five_calls_in_one_graph(hd):  # noqa: F811
    """append, attention, weights, selection and moves captured once and replayed with other lengths and inputs, next
    to the same steps called one by one: equal bit for bit, state and outputs."""
    a, b = Server(1), Server(1)
    b.take([0] * 5, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(hd)
        b.kv.copy_(b.new)
    for i, n in enumerate(STEPS):
        a.take(n, 100 + i)
        a.step(hd)
        a.kv.copy_(a.new)
        b.take(n, 100 + i)
        graph.replay()
        hd.hcadsa_check_device_error()
        for x, y in zip(a.state(), b.state()):
            assert same(x, y), (i, x.shape)
    assert (a.moves >= 0).any() and a.kv.tolist() == [96, 96, 96, 96, 63]  # 1 + 1 + 7 + 0 + 1 + 1 + 52 rows


def test_five_calls_on_a_stream(hd):  # noqa: F811
    """The same on a stream given to the calls, while the current one is busy."""
    a, b = Server(2), Server(2)
    s = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    for i, n in enumerate(STEPS):
        a.take(n, 200 + i)
        a.step(hd)
        a.kv.copy_(a.new)
        b.take(n, 200 + i)
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            busy = busy @ busy * 1e-3
        b.step(hd, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        b.kv.copy_(b.new)
        for x, y in zip(a.state(), b.state()):
            assert same(x, y), (i, x.shape)
    hd.hcadsa_check_device_error()


FIRST_CALLS_CAPTURED = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import sparse_attention_hca_b200 as hd
from test_gpu_mla_serving import STEPS, Server, same
a, b = Server(1), Server(1)
b.take(STEPS[0], 100)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    b.step(hd)
graph.replay()
a.take(STEPS[0], 100)
a.step(hd)
hd.hcadsa_check_device_error()
assert all(same(x, y) for x, y in zip(a.state(), b.state()))
print("captured")
"""


def test_first_calls_of_a_process_are_captured(hd):  # noqa: F811
    """A process whose first calls of the library are captured: what is set up once is set up there."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED.format(root=ROOT)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


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
