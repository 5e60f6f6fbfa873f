"""GPU tests of the paged cache of the full-context (MLA) layers: mla_cache_append,
mla_paged_attn_fwd, mla_paged_attn_mass, mla_evict_select and mla_cache_move against plain
implementations in 64 bits, written from the definitions.

Tolerances, from the arithmetic (u = 2^-8 is half a bf16 step, relative):
  scores  an fp32 sum of 256 exact products, any order, adds that truncate: off by at most
          d = 256 * 2^-23 * max_s scale * sum_c |q_c k_sc|, which is the relative error of a weight
          (twice that once divided by the sum of the weights, itself off by as much);
  O       weights rounded to bf16 (u each), then O rounded: |err| <= u |O| + (u + 2 d + 2^-18) A,
          A = sum_s p_s |v_s| (the 2^-18 covers the exponential, the fp32 sums and 1/l), times
          1 + u for the product of the two roundings;
  lse     d + 2^-18 + 2^-22 |lse| + (rows) 2^-24;
  mass    a sum of N positive weights: relative 2 d + 2^-18 + 2^-21 max(|x| + |lse|) + N 2^-24.
Everything that is copied or selected has to be equal."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
bf, f32, f64, i32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
D = 256
U = 2.0 ** -8


@pytest.fixture(scope="module")
def hd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_hca_b200 import build

    build.build()
    import sparse_attention_hca_b200 as m

    return m


class Cache:
    """Pools in which everything but the sequences' rows is NaN (K, V), and a batch over them."""

    def __init__(self, q_len, kv_len, Hq=64, Hkv=1, page=64, seed=0, interleaved=False, extra_pages=3, width=None,
                 pad=0, sigma=1.0, fused=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.q_len, self.kv, self.Hq, self.Hkv, self.page = g, list(q_len), list(kv_len), Hq, Hkv, page
        B = len(q_len)
        width = width or max(1, max(-(-n // page) for n in kv_len))
        n_pages = B * width + extra_pages
        nan = float("nan")
        if interleaved:
            pool = torch.full((n_pages, 2, page, Hkv, D), nan, dtype=bf, device="cuda")
            self.K, self.V = pool[:, 0], pool[:, 1]
        else:
            self.K = torch.full((n_pages, page, Hkv, D), nan, dtype=bf, device="cuda")
            self.V = torch.full((n_pages, page, Hkv, D), nan, dtype=bf, device="cuda")
        self.table = torch.randperm(n_pages, generator=g, device="cuda")[: B * width].reshape(B, width).to(i32)
        self.cu = torch.tensor([0] + list(torch.tensor(q_len).cumsum(0)), dtype=i32, device="cuda")
        self.kv_len = torch.tensor(kv_len, dtype=i32, device="cuda")
        T = sum(q_len) + pad
        if fused:  # slices of one fused projection
            qkv = self.rand(T, Hq + 2 * Hkv, D) * sigma
            self.q, self.k_new, self.v_new = qkv[:, :Hq], qkv[:, Hq : Hq + Hkv], qkv[:, Hq + Hkv :]
        else:
            self.q = self.rand(T, Hq, D) * sigma
        for b in range(B):
            at = self.rows(b)
            self.K[at] = self.rand(self.kv[b], Hkv, D)
            self.V[at] = self.rand(self.kv[b], Hkv, D)

    def rand(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda").to(bf)

    def rows(self, b, n=None):
        i = torch.arange(self.kv[b] if n is None else n, device="cuda")
        return self.table[b].long()[i // self.page], i % self.page

    def args(self):
        return self.K, self.V, self.table, self.cu, self.kv_len


def oracle(c, scale=None, lse_in=None):
    """Per sequence: O, A, lse, the score bound d, and with lse_in the mass and its bound."""
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    T = c.q.shape[0]
    grp = c.Hq // c.Hkv
    O = torch.zeros((T, c.Hq, D), dtype=f64, device="cuda")
    A = torch.zeros_like(O)
    lse = torch.full((T, c.Hq), -math.inf, dtype=f64, device="cuda")
    d = torch.zeros((T, c.Hq), dtype=f64, device="cuda")
    mass = torch.zeros(c.K.shape[:3], dtype=f64, device="cuda")
    tol = torch.zeros_like(mass)
    t = 0
    for b, n in enumerate(c.q_len):
        if n and c.kv[b]:
            k, v = c.K[c.rows(b)].double(), c.V[c.rows(b)].double()
            q = c.q[t : t + n].double()
            see = torch.arange(c.kv[b], device="cuda")[None] <= (c.kv[b] - n + torch.arange(n, device="cuda"))[:, None]
            for h in range(c.Hq):
                x = scale * q[:, h] @ k[:, h // grp].T
                big = 256 * 2.0 ** -23 * (scale * q[:, h].abs() @ k[:, h // grp].abs().T)
                x = x.masked_fill(~see, -math.inf)
                lse[t : t + n, h] = torch.logsumexp(x, 1)
                p = torch.softmax(x, 1).nan_to_num(0.0)
                O[t : t + n, h] = p @ v[:, h // grp]
                A[t : t + n, h] = p @ v[:, h // grp].abs()
                d[t : t + n, h] = big.masked_fill(~see, 0.0).amax(1)
                if lse_in is not None:
                    li = lse_in[t : t + n, h].double()
                    w = torch.exp(x - li[:, None]).masked_fill(~see, 0.0)
                    one = 2 * big + 2.0 ** -18 + 2.0 ** -21 * (x.abs() + li[:, None].abs()) + n * grp * 2.0 ** -24
                    at = c.rows(b)
                    mass[at[0], at[1], h // grp] += w.sum(0)
                    tol[at[0], at[1], h // grp] += (w * one.masked_fill(~see, 0.0)).sum(0)
        t += n
    return O, A, lse, d, mass, tol


def check_attn(c, O, lse, ref, what):
    o64, A, l64, d = ref[:4]
    n = sum(c.q_len)
    bound = (1 + U) * (U * o64.abs() + (U + 2 * d[..., None] + 2.0 ** -18) * A) + 1e-30
    err = (O.double() - o64).abs()[:n]
    assert torch.isfinite(O[:n].float()).all(), what
    assert (err <= bound[:n]).all(), (what, (err / bound[:n]).max().item())
    empty = l64 == -math.inf
    assert torch.equal(lse[:n] == -math.inf, empty[:n]), what
    fine = ~empty[:n]
    lb = (d + 2.0 ** -18 + 2.0 ** -22 * l64.abs() + max(c.kv) * 2.0 ** -24)[:n][fine]
    le = (lse.double() - l64).abs()[:n][fine]
    assert (le <= lb).all(), (what, (le / lb).max().item())
    assert (O[:n][empty[:n]] == 0).all(), what


CASES = {
    "one_token_one_row": dict(q_len=[1], kv_len=[1]),
    "decode_ragged": dict(q_len=[1] * 5, kv_len=[1, 17, 128, 129, 1000], page=16),
    "decode_gqa": dict(q_len=[1, 1, 1], kv_len=[300, 64, 511], Hq=32, Hkv=4, page=32),
    "decode_mha": dict(q_len=[1, 1], kv_len=[255, 257], Hq=16, Hkv=16, page=128),
    "decode_group128": dict(q_len=[1, 2], kv_len=[130, 259], Hq=128, Hkv=1, page=64),
    "decode_group128_one_token_each": dict(q_len=[1, 1, 1], kv_len=[130, 2000, 64], Hq=128, Hkv=1, page=32),
    "decode_two_groups_of_128": dict(q_len=[1, 1], kv_len=[700, 129], Hq=256, Hkv=2, page=16),
    "one_row_per_token": dict(q_len=[1] * 3, kv_len=[77, 400, 1000], Hq=3, Hkv=3, page=16),
    "long_chunk": dict(q_len=[1100], kv_len=[2300], page=128),
    "short_tail_tiles": dict(q_len=[5, 5, 5, 5], kv_len=[129, 257, 145, 17], page=16, Hq=32),
    "prompt_from_nothing": dict(q_len=[300], kv_len=[300]),
    "chunk_odd": dict(q_len=[37, 129], kv_len=[700, 129], page=16),
    "chunk_gqa_fused_pool": dict(q_len=[65, 1, 200], kv_len=[400, 33, 777], Hq=8, Hkv=2, page=256, interleaved=True),
    "chunk_one_head": dict(q_len=[513, 3], kv_len=[900, 3], Hq=1, Hkv=1, page=64),
    "mixed": dict(q_len=[1, 77, 1, 1, 40], kv_len=[2500, 1290, 1, 640, 40], page=32, interleaved=True),
    "sequences_without_tokens": dict(q_len=[0, 5, 0, 1, 0], kv_len=[50, 70, 0, 9, 3], page=16),
    "rows_that_see_nothing": dict(q_len=[9, 130, 2], kv_len=[4, 0, 300], page=16),
    "padded_rows": dict(q_len=[3, 20], kv_len=[150, 20], pad=50, page=1024),
    "fused_projection": dict(q_len=[50, 1], kv_len=[333, 200], Hq=16, Hkv=2, fused=True),
    "sharp": dict(q_len=[33, 1], kv_len=[500, 3000], sigma=8.0),
    "many_sequences": dict(q_len=[1, 2, 0, 3] * 120, kv_len=[40, 2, 5, 177] * 120, Hq=16, page=16),
    "many_prompts": dict(q_len=[4, 0, 9, 1, 40] * 100, kv_len=[300, 10, 9, 150, 700] * 100, Hq=16, page=32),
    "short_row_tiles": dict(q_len=[256], kv_len=[1024]),
    "short_and_long_row_tiles": dict(q_len=[100, 64, 31], kv_len=[1200, 5000, 31], Hq=32, Hkv=2, page=128),
    "long_decode": dict(q_len=[1, 4], kv_len=[40000, 20001], page=64),
}


@pytest.mark.parametrize("name", list(CASES))
def test_attention_and_mass(hd, name):
    c = Cache(seed=len(name), **CASES[name])
    T = c.q.shape[0]
    O = torch.full((T, c.Hq, D), 7.0, dtype=bf, device="cuda")
    lse = torch.full((T, c.Hq), 7.0, device="cuda")
    hd.mla_paged_attn_fwd(c.q, *c.args(), O=O, lse=lse, return_lse=True)
    hd.hcadsa_check_device_error()
    ref = oracle(c, lse_in=lse)
    check_attn(c, O, lse, ref, name)
    n = sum(c.q_len)
    assert (O[n:] == 7).all() and (lse[n:] == 7).all()  # rows behind the last sequence
    start = torch.rand(c.K.shape[:3], generator=c.g, device="cuda")
    mass = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse, mass=start.clone())
    hd.hcadsa_check_device_error()
    err = (mass.double() - start.double() - ref[4]).abs()
    bound = ref[5] + 2.0 ** -23 * (start.double() + ref[4])
    assert (err <= bound).all(), (name, (err / bound.clamp_min(1e-30)).max().item())
    assert torch.equal(mass[ref[4] == 0], start[ref[4] == 0])
    # all the weight of the rows that see something
    total = (lse[:n] > -math.inf).sum().item()
    assert abs(ref[4].sum().item() - total) <= 1e-2 * total + 1e-9
    # the same call again gives the same bits
    O2, lse2 = hd.mla_paged_attn_fwd(c.q, *c.args(), return_lse=True)
    assert torch.equal(O2[:n], O[:n]) and torch.equal(lse2[:n], lse[:n])
    m2 = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse, mass=start.clone())
    assert torch.equal(m2, mass)


def test_scale_and_defaults(hd):
    c = Cache([20], [150], Hq=16, seed=3)
    O, lse = hd.mla_paged_attn_fwd(c.q, *c.args(), scale=0.01, return_lse=True)
    check_attn(c, O, lse, oracle(c, 0.01), "scale")
    only = hd.mla_paged_attn_fwd(c.q, *c.args(), scale=0.01)
    assert torch.equal(only, O)
    mass = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse, scale=0.01)
    ref = oracle(c, 0.01, lse_in=lse)
    assert ((mass.double() - ref[4]).abs() <= ref[5] + 2.0 ** -23 * ref[4]).all()


def test_weights_equal_keys(hd):
    """Equal keys: uniform weights, so O is the mean of the visible values and mass is known in closed form."""
    c = Cache([4], [260], Hq=64, seed=5)
    c.K[c.rows(0)] = 0.5
    O, lse = hd.mla_paged_attn_fwd(c.q, *c.args(), return_lse=True)
    mass = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse)
    got = mass[c.rows(0)][:, 0].double()
    want = torch.zeros(260, dtype=f64, device="cuda")
    for t in range(4):
        want[: 257 + t] += 64.0 / (257 + t)
    assert ((got - want).abs() <= 1e-4 * want).all()
    check_attn(c, O, lse, oracle(c), "equal keys")


def test_pages_beyond_2_31_elements(hd):
    """Pools of more than 2^31 elements: the sequences' pages are the last ones."""
    page, n_pages = 64, 140000  # 2.29e9 elements in each pool
    K = torch.empty((n_pages, page, 1, D), dtype=bf, device="cuda")
    V = torch.empty((n_pages, page, 1, D), dtype=bf, device="cuda")
    c = Cache([3, 1], [200, 77], seed=9)
    width = c.table.shape[1]
    table = (n_pages - 1 - torch.arange(2 * width, device="cuda")).reshape(2, width).to(i32)
    K[table.long()], V[table.long()] = c.K[c.table.long()], c.V[c.table.long()]
    O, lse = hd.mla_paged_attn_fwd(c.q, K, V, table, c.cu, c.kv_len, return_lse=True)
    check_attn(c, O, lse, oracle(c), "far pages")
    mass = hd.mla_paged_attn_mass(c.q, K, table, c.cu, c.kv_len, lse)
    near = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse)
    assert torch.equal(mass[table.long()], near[c.table.long()])
    new = c.rand(4, 1, D)
    hd.mla_cache_append(new, new, K, V, table, c.cu, c.kv_len, mass=mass)
    at = torch.arange(197, 200, device="cuda")
    assert torch.equal(K[table[0].long()[at // page], at % page], new[:3])
    moves = torch.tensor([[[[199, 3]]], [[[-1, -1]]]], dtype=i32, device="cuda")
    hd.mla_cache_move(moves, K, V, table, mass=mass)
    hd.hcadsa_check_device_error()
    assert torch.equal(V[table[0, 0], 3], new[2])


@pytest.mark.parametrize("Hkv,page,fused", [(1, 16, False), (4, 64, True), (3, 128, False)])
def test_append(hd, Hkv, page, fused):
    c = Cache([5, 0, 1, 70], [5, 40, 100, 333], Hq=4 * Hkv, Hkv=Hkv, page=page, seed=Hkv, pad=9, fused=True)
    k, v = (c.k_new, c.v_new) if fused else (c.k_new.contiguous(), c.v_new.contiguous())
    seen = c.kv_len + torch.tensor([0, 3, 1000, 5], dtype=i32, device="cuda")
    pos = torch.full(c.K.shape[:3], -5, dtype=i32, device="cuda")
    mass = torch.full(c.K.shape[:3], 3.0, device="cuda")
    want = [x.clone() for x in (c.K, c.V, pos, mass)]
    t = 0
    for b, n in enumerate(c.q_len):
        i = torch.arange(c.kv[b] - n, c.kv[b], device="cuda")
        at = c.table[b].long()[i // page], i % page
        want[0][at], want[1][at] = k[t : t + n], v[t : t + n]
        want[2][at] = (seen[b] - n + torch.arange(n, device="cuda")).to(i32)[:, None]
        want[3][at] = 0.0
        t += n
    hd.mla_cache_append(k, v, c.K, c.V, c.table, c.cu, c.kv_len, seen=seen, pos=pos, mass=mass)
    hd.hcadsa_check_device_error()
    for a, w in zip((c.K, c.V, pos, mass), want):
        assert torch.equal(a.view(torch.int16) if a.dtype == bf else a, w.view(torch.int16) if w.dtype == bf else w)
    # without seen the position is the row number; pos and mass are optional
    hd.mla_cache_append(k, v, c.K, c.V, c.table, c.cu, c.kv_len, pos=pos)
    at = c.table[3].long()[332 // page], 332 % page
    assert (pos[at] == 332).all()
    hd.mla_cache_append(k, v, c.K, c.V, c.table, c.cu, c.kv_len)


def select_oracle(mass, pos, table, kv, seen, budget, sink, recent, page):
    """Python lists, straight from the definition: per (sequence, head) the (from, to) pairs."""
    out = []
    for b, n in enumerate(kv):
        per = []
        for h in range(mass.shape[2]):
            rows = [(table[b][i // page], i % page, h) for i in range(n)]
            m = [float(mass[r]) for r in rows]
            ps = [int(pos[r]) for r in rows]
            safe = [p < sink or p >= seen[b] - recent for p in ps]
            order = sorted(range(n), key=lambda i: (not safe[i], -m[i] if m[i] == m[i] else -math.inf, i))
            if any(x != x for x in m):  # NaN counts as more than +inf
                order = sorted(range(n), key=lambda i: (not safe[i], m[i] == m[i], -m[i] if m[i] == m[i] else 0, i))
            keep = set(order[:budget]) if n > budget else set(range(n))
            late = [i for i in range(budget, n) if i in keep]
            free = [i for i in range(min(n, budget)) if i not in keep]
            assert len(late) == len(free)
            per.append(list(zip(late, free)))
        out.append(per)
    return out


SELECT = {
    "one_over": dict(kv=[17], budget=16, sink=1, recent=4, page=16),
    "budget_one": dict(kv=[200, 1], budget=1, sink=0, recent=0, page=16),
    "ragged": dict(kv=[0, 5, 64, 65, 700, 1031], budget=64, sink=4, recent=16, page=32, Hkv=2),
    "ties": dict(kv=[3000, 2999], budget=1000, sink=2, recent=100, page=64, levels=3),
    "all_equal": dict(kv=[5000], budget=1234, sink=0, recent=0, page=64, levels=1),
    "all_protected": dict(kv=[900], budget=300, sink=100, recent=200, page=64),
    "cluster": dict(kv=[40000, 33000], budget=9000, sink=8, recent=1000, page=128, Hkv=2),
    "cluster_ties": dict(kv=[50001], budget=25000, sink=8, recent=1000, page=16, levels=2),
    "large_cluster": dict(kv=[70001, 66000], budget=30000, sink=8, recent=1000, page=64, levels=100),
    "many_lists": dict(kv=[300, 17, 2100] * 30, budget=100, sink=4, recent=20, page=16, Hkv=2, levels=50),
    "many_longer_lists": dict(kv=[9000, 4000] * 40, budget=300, sink=4, recent=20, page=64, levels=200),
    "special_values": dict(kv=[2000], budget=700, sink=4, recent=10, page=64, special=True),
    "wide_table": dict(kv=[300, 100], budget=100, sink=1, recent=2, page=16, width=4000),
    "nothing_to_do": dict(kv=[30, 64], budget=64, sink=1, recent=2, page=64, width=2),
    "table_within_budget": dict(kv=[30, 64], budget=200, sink=1, recent=2, page=64, width=2),
}


@pytest.mark.parametrize("name", list(SELECT))
def test_select_and_move(hd, name):
    a = dict(Hkv=1, levels=0, special=False, width=None)
    a.update(SELECT[name])
    kv, page, Hkv, budget = a["kv"], a["page"], a["Hkv"], a["budget"]
    g = torch.Generator().manual_seed(len(name))
    width = a["width"] or max(-(-n // page) for n in kv)
    n_pages = len(kv) * width + 2
    table = torch.randperm(n_pages, generator=g)[: len(kv) * width].reshape(len(kv), width).to(i32)
    mass = torch.randn((n_pages, page, Hkv), generator=g).exp()
    if a["levels"]:
        mass = torch.randint(0, a["levels"], mass.shape, generator=g).float()
    if a["special"]:
        pick = torch.randint(0, 8, mass.shape, generator=g)
        for i, x in enumerate((math.inf, -math.inf, math.nan, 0.0, -0.0, -1.0, 1e-42)):
            mass[pick == i] = x
    seen = [n + 57 for n in kv]
    pos = torch.zeros((n_pages, page, Hkv), dtype=i32)
    for b, n in enumerate(kv):
        for h in range(Hkv):
            p = torch.randperm(n + 57, generator=g)[:n].to(i32)
            i = torch.arange(n)
            pos[table[b].long()[i // page], i % page, h] = p
    K = torch.randn((n_pages, page, Hkv, D), generator=g).to(bf)
    V = torch.randn((n_pages, page, Hkv, D), generator=g).to(bf)
    want = select_oracle(mass.numpy(), pos.numpy(), table.tolist(), kv, seen, budget, a["sink"], a["recent"], page)
    dev = [x.cuda() for x in (mass, pos, table, torch.tensor(kv, dtype=i32), torch.tensor(seen, dtype=i32))]
    moves, new_len = hd.mla_evict_select(*dev, budget, n_sink=a["sink"], n_recent=a["recent"])
    hd.hcadsa_check_device_error()
    assert new_len.tolist() == [min(n, budget) for n in kv]
    assert moves.shape[2] == max(0, min(budget, width * page - budget))
    for b in range(len(kv)):
        for h in range(Hkv):
            w = want[b][h]
            assert moves[b, h, : len(w)].tolist() == [list(x) for x in w], (name, b, h)
            assert (moves[b, h, len(w) :] == -1).all()
    Kd, Vd, pd, md = K.cuda(), V.cuda(), dev[1].clone(), dev[0].clone()
    hd.mla_cache_move(moves, Kd, Vd, dev[2], pos=pd, mass=md)
    hd.hcadsa_check_device_error()
    for got, ref in ((Kd, K), (Vd, V), (pd, pos), (md, mass)):
        ref = ref.clone()
        for b in range(len(kv)):
            for h in range(Hkv):
                if want[b][h]:
                    f, t = torch.tensor(want[b][h]).unbind(1)
                    tb = table[b].long()
                    ref[tb[t // page], t % page, h] = ref[tb[f // page], f % page, h]
        same = (got.cpu() == ref) | ((got.cpu() != got.cpu()) & (ref != ref))
        assert same.all(), name
    again, _ = hd.mla_evict_select(*dev, budget, n_sink=a["sink"], n_recent=a["recent"])
    assert torch.equal(again, moves)


@pytest.mark.parametrize("n, lists", [(420001, 1), (900001, 1), (420001, 8)])
def test_select_rows_read_again(hd, n, lists):
    """Caches longer than their clusters' shared memory (44K rows per CTA, 16 CTAs for few lists, 8 for
    more) are read from memory in every pass.  The lists are the same sequence, several times."""
    page, budget = 1024, 100000
    width = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randperm(width, generator=g, device="cuda").to(i32)[None].repeat(lists, 1)
    mass = torch.randint(0, 1000, (width, page, 1), generator=g, device="cuda").float()
    pos = torch.zeros((width, page, 1), dtype=i32, device="cuda")
    i = torch.arange(n, device="cuda")
    at = table[0].long()[i // page], i % page
    pos[at] = i.to(i32)[:, None]
    kv = torch.tensor([n] * lists, dtype=i32, device="cuda")
    moves, _ = hd.mla_evict_select(mass, pos, table, kv, None, budget, n_sink=16, n_recent=5000)
    hd.hcadsa_check_device_error()
    m = mass[at][:, 0].clone()
    m[:16] = math.inf
    m[n - 5000 :] = math.inf
    keep = torch.zeros(n, dtype=torch.bool, device="cuda")
    keep[m.argsort(descending=True, stable=True)[:budget]] = True
    late, free = keep[budget:].nonzero()[:, 0] + budget, (~keep[:budget]).nonzero()[:, 0]
    for b in range(lists):
        assert torch.equal(moves[b, 0, : len(late), 0].long(), late)
        assert torch.equal(moves[b, 0, : len(free), 1].long(), free)
        assert (moves[b, 0, len(late) :] == -1).all()


def test_device_errors_are_recorded_and_stay_inside(hd):
    """Tables and lengths out of range: recorded, and the other sequences keep their results."""
    c = Cache([4, 3, 2], [200, 150, 90], seed=11, Hq=16)
    good = hd.mla_paged_attn_fwd(c.q, *c.args())
    table = c.table.clone()
    table[1, 0], table[1, 1] = -1, 1 << 29
    n_err = 0

    def failing(call):
        nonlocal n_err
        r = call()
        with pytest.raises(hd.HcaDsaError, match="DEVICE_BOUNDS"):
            hd.hcadsa_check_device_error()
        n_err += 1
        return r

    O = failing(lambda: hd.mla_paged_attn_fwd(c.q, c.K, c.V, table, c.cu, c.kv_len))
    assert torch.equal(O[:4], good[:4]) and torch.equal(O[7:], good[7:]) and torch.isfinite(O.float()).all()
    lse = torch.zeros((9, 16), device="cuda")
    failing(lambda: hd.mla_paged_attn_mass(c.q, c.K, table, c.cu, c.kv_len, lse))
    new = c.rand(9, 1, D)
    K0 = c.K.clone()
    bad_end = c.table.clone()
    bad_end[1, 149 // 64] = 1 << 30
    failing(lambda: hd.mla_cache_append(new, new, c.K, c.V, bad_end, c.cu, c.kv_len))
    at = c.table[1].long()
    assert torch.equal(c.K[at].view(torch.int16), K0[at].view(torch.int16))
    moves = torch.tensor([[[[5, 1 << 20]]], [[[3, 2]]], [[[-1, 4]]]], dtype=i32, device="cuda")
    failing(lambda: hd.mla_cache_move(moves, c.K, c.V, table))
    mass = torch.zeros(c.K.shape[:3], device="cuda")
    pos = torch.zeros(c.K.shape[:3], dtype=i32, device="cuda")
    failing(lambda: hd.mla_evict_select(mass, pos, table, c.kv_len, None, 64))
    good = hd.mla_paged_attn_fwd(c.q, *c.args())  # the other sequences' appends and moves were made
    for kv in ([200, 1 << 30, 90], [200, -7, 90]):
        O = failing(lambda: hd.mla_paged_attn_fwd(c.q, c.K, c.V, c.table, c.cu, torch.tensor(kv, dtype=i32, device="cuda")))
        assert torch.equal(O[:2], good[:2])
    for cu in ([0, 4, 2, 9], [0, 4, 7, 1 << 30], [-3, 4, 7, 9]):
        failing(lambda: hd.mla_paged_attn_fwd(c.q, c.K, c.V, c.table, torch.tensor(cu, dtype=i32, device="cuda"), c.kv_len))
    assert n_err == 10
    assert torch.equal(hd.mla_paged_attn_fwd(c.q, *c.args())[:2], good[:2])
    hd.hcadsa_check_device_error()


def test_other_stream_and_graph(hd):
    """A call on a given stream, and the calls captured into a graph and replayed on new inputs and lengths."""
    c = Cache([1, 30], [500, 260], seed=13, width=10)
    want, wl = hd.mla_paged_attn_fwd(c.q, *c.args(), return_lse=True)
    wm = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, wl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    O, lse = hd.mla_paged_attn_fwd(c.q, *c.args(), return_lse=True, stream=s)
    mass = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(O, want) and torch.equal(lse, wl) and torch.equal(mass, wm)
    graph = torch.cuda.CUDAGraph()
    q, kv, cu = c.q.clone(), c.kv_len.clone(), c.cu.clone()
    with torch.cuda.graph(graph):
        gO, gl = hd.mla_paged_attn_fwd(q, c.K, c.V, c.table, cu, kv, return_lse=True)
        gm = hd.mla_paged_attn_mass(q, c.K, c.table, cu, kv, gl)
    graph.replay()
    assert torch.equal(gO, want) and torch.equal(gm, wm)
    c2 = Cache([7, 24], [123, 300], seed=14, width=10)
    c.K.copy_(c2.K), c.V.copy_(c2.V), c.table.copy_(c2.table)
    q.copy_(c2.q), kv.copy_(c2.kv_len), cu.copy_(c2.cu)
    graph.replay()
    want2, wl2 = hd.mla_paged_attn_fwd(c2.q, *c2.args(), return_lse=True)
    assert torch.equal(gO, want2) and torch.equal(gl, wl2)
    assert torch.equal(gm, hd.mla_paged_attn_mass(c2.q, c2.K, c2.table, c2.cu, c2.kv_len, wl2))
    hd.hcadsa_check_device_error()


def test_unaligned_outputs_and_workspaces(hd):
    """O on a 16-byte boundary only, pos and mass on a 4-byte one, a caller's workspace, and the refusals of short or
    misaligned ones."""
    c = Cache([3, 70], [500, 140], seed=17, Hq=16)
    want, wl = hd.mla_paged_attn_fwd(c.q, *c.args(), return_lse=True)
    buf = torch.zeros(73 * 16 * D + 8, dtype=bf, device="cuda")
    O = buf[8:].view(73, 16, D)
    need = hd.lib().mla_paged_attn_fwd_workspace_size(2, 73, 16, 1)
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    hd.mla_paged_attn_fwd(c.q, *c.args(), O=O, workspace=ws[:need])
    assert torch.equal(O, want) and (buf[:8] == 0).all()
    for bad, what in ((ws[: need - 1], "WORKSPACE"), (ws[16:], "ALIGN")):
        with pytest.raises(hd.HcaDsaError, match=what):
            hd.mla_paged_attn_fwd(c.q, *c.args(), workspace=bad)
    need = hd.lib().mla_paged_attn_mass_workspace_size(2, 73, 16, 1)
    with pytest.raises(hd.HcaDsaError, match="WORKSPACE"):
        hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, wl, workspace=ws[: need - 1])
    mass = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, wl, workspace=ws[:need])
    pos = torch.arange(mass.numel(), dtype=i32, device="cuda").view(mass.shape)
    a, _ = hd.mla_evict_select(mass, pos, c.table, c.kv_len, None, 100, n_sink=2, n_recent=5)
    off = [torch.cat([x.new_zeros(1), x.flatten()])[1:].view(x.shape) for x in (mass, pos)]
    b, _ = hd.mla_evict_select(*off, c.table, c.kv_len, None, 100, n_sink=2, n_recent=5)
    assert torch.equal(a, b)
    hd.hcadsa_check_device_error()


def test_two_calls_at_once(hd):
    """Calls on two streams that overlap, each with its own outputs and workspace."""
    cs = [Cache([1] * 6, [3000, 50, 777, 4096, 1, 129], seed=31), Cache([260, 1], [900, 2000], seed=32, page=16)]
    want = []
    for c in cs:
        O, lse = hd.mla_paged_attn_fwd(c.q, *c.args(), return_lse=True)
        want.append((O, lse, hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (c, s) in enumerate(zip(cs, streams)):
            O, lse = hd.mla_paged_attn_fwd(c.q, *c.args(), return_lse=True, stream=s)
            got[i].append((O, lse, hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse, stream=s)))
    torch.cuda.synchronize()
    hd.hcadsa_check_device_error()
    for w, many in zip(want, got):
        for g in many:
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_shared_pages(hd):
    """Two sequences that share their first pages: attention reads them for both, and a shared row's mass is the sum."""
    c = Cache([1, 20], [200, 200], seed=41, page=16)
    c.table[1, :8] = c.table[0, :8]
    at = c.rows(1)
    c.K[at[0][128:], at[1][128:]] = c.rand(72, 1, D)
    O, lse = hd.mla_paged_attn_fwd(c.q, *c.args(), return_lse=True)
    ref = oracle(c, lse_in=lse)
    check_attn(c, O, lse, ref, "shared pages")
    mass = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse)
    assert ((mass.double() - ref[4]).abs() <= ref[5] + 2.0 ** -22 * ref[4]).all()
    hd.hcadsa_check_device_error()


def test_many_empty_sequences(hd):
    """More sequences than threads in a block, most of them without tokens or rows."""
    n = 1500
    q = [3 if b % 401 == 7 else 0 for b in range(n)]
    kv = [130 if q[b] else (b % 5) * 3 for b in range(n)]
    c = Cache(q, kv, Hq=16, page=16, seed=43, width=9)
    O, lse = hd.mla_paged_attn_fwd(c.q, *c.args(), return_lse=True)
    ref = oracle(c, lse_in=lse)
    check_attn(c, O, lse, ref, "many")
    mass = hd.mla_paged_attn_mass(c.q, c.K, c.table, c.cu, c.kv_len, lse)
    assert ((mass.double() - ref[4]).abs() <= ref[5] + 2.0 ** -23 * ref[4]).all()
    none = hd.mla_paged_attn_fwd(c.q, c.K, c.V, c.table, torch.zeros_like(c.cu), c.kv_len, O=torch.ones_like(O))
    assert (none == 1).all()
    hd.hcadsa_check_device_error()


def test_empty_calls(hd):
    c = Cache([0, 0], [5, 3], seed=1, Hq=16)
    q = c.q[:0]
    O, lse = hd.mla_paged_attn_fwd(q, *c.args(), return_lse=True)
    assert O.shape == (0, 16, D) and lse.shape == (0, 16)
    assert (hd.mla_paged_attn_mass(q, c.K, c.table, c.cu, c.kv_len, lse) == 0).all()
    hd.mla_cache_append(c.rand(0, 1, D), c.rand(0, 1, D), c.K, c.V, c.table, c.cu, c.kv_len)
    none = torch.zeros((0, 4), dtype=i32, device="cuda")
    hd.mla_paged_attn_fwd(c.rand(4, 16, D), c.K, c.V, none, torch.zeros(1, dtype=i32, device="cuda"),
                          torch.zeros(0, dtype=i32, device="cuda"))
    hd.hcadsa_check_device_error()


def test_serving_loop(hd):
    """Chunks and single tokens through append -> attention -> mass -> eviction, the caches held to a budget, against
    the same loop on lists of rows in 64 bits."""
    Hq, Hkv, page, budget, sink, recent, B = 16, 2, 16, 96, 2, 20, 3
    g = torch.Generator(device="cuda").manual_seed(21)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(bf)  # noqa: E731
    width = 12
    n_pages = B * width
    K, V = torch.full((2, n_pages, page, Hkv, D), math.nan, dtype=bf, device="cuda").unbind(0)
    pos = torch.zeros((n_pages, page, Hkv), dtype=i32, device="cuda")
    mass = torch.zeros((n_pages, page, Hkv), device="cuda")
    table = torch.randperm(n_pages, generator=g, device="cuda").reshape(B, width).to(i32)
    kv, seen = torch.zeros(B, dtype=i32, device="cuda"), torch.zeros(B, dtype=i32, device="cuda")
    mine = [[[] for _ in range(Hkv)] for _ in range(B)]  # rows: [k, v, pos] in cache order
    for step, n in enumerate([[60, 0, 90], [50, 40, 1], [1, 1, 1], [33, 70, 80], [1, 1, 1], [0, 2, 60]]):
        T = sum(n)
        q, k, v = rnd(T, Hq, D), rnd(T, Hkv, D), rnd(T, Hkv, D)
        cu = torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=i32, device="cuda")
        add = torch.tensor(n, dtype=i32, device="cuda")
        kv, seen = kv + add, seen + add
        hd.mla_cache_append(k, v, K, V, table, cu, kv, seen=seen, pos=pos, mass=mass)
        O, lse = hd.mla_paged_attn_fwd(q, K, V, table, cu, kv, return_lse=True)
        hd.mla_paged_attn_mass(q, K, table, cu, kv, lse, mass=mass)
        t = 0
        for b in range(B):
            for h in range(Hkv):
                rows = mine[b][h]
                p0 = int(seen[b]) - n[b]
                rows += [[k[t + i, h], v[t + i, h], p0 + i] for i in range(n[b])]
                assert len(rows) == int(kv[b])
                if not n[b]:
                    continue
                kk = torch.stack([r[0] for r in rows]).double()
                vv = torch.stack([r[1] for r in rows]).double()
                for hq in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                    x = q[t : t + n[b], hq].double() @ kk.T / 16.0
                    see = torch.arange(len(rows), device="cuda")[None] <= torch.arange(
                        len(rows) - n[b], len(rows), device="cuda")[:, None]
                    p = torch.softmax(x.masked_fill(~see, -math.inf), 1)
                    o = p @ vv
                    bound = (1 + U) * (U * o.abs() + (U + 2.0 ** -9) * (p @ vv.abs()))
                    assert ((O[t : t + n[b], hq].double() - o).abs() <= bound).all(), (step, b, hq)
            t += n[b]
        # eviction by the accumulated masses (read back: the selection has to be exact on them)
        moves, new = hd.mla_evict_select(mass, pos, table, kv, seen, budget, n_sink=sink, n_recent=recent)
        want = select_oracle(mass.cpu().numpy(), pos.cpu().numpy(), table.tolist(), kv.tolist(), seen.tolist(), budget,
                             sink, recent, page)
        hd.mla_cache_move(moves, K, V, table, pos=pos, mass=mass)
        kv = new
        for b in range(B):
            i = torch.arange(int(kv[b]), device="cuda")
            at = table[b].long()[i // page], i % page
            for h in range(Hkv):
                w = want[b][h]
                assert moves[b, h, : len(w)].tolist() == [list(x) for x in w]
                rows = mine[b][h]
                for f, to in w:
                    rows[to] = rows[f]
                del rows[budget:]
                assert pos[at][:, h].tolist() == [r[2] for r in rows]
                if rows:
                    assert torch.equal(K[at][:, h], torch.stack([r[0] for r in rows]))
                    assert torch.equal(V[at][:, h], torch.stack([r[1] for r in rows]))
                    kept = pos[at][:, h]
                    assert all(p in kept.tolist() for p in range(min(sink, int(seen[b]))))
    hd.hcadsa_check_device_error()
