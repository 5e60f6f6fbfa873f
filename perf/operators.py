"""Measured cases of the paged-cache operators of the full-context (MLA) layers: 256-wide heads, bf16 K and V
rows in pages, a chunk of new tokens per sequence.

  append   writes a chunk's new rows to the ends of their sequences' caches, with their positions
  attn     attention of the chunk's query heads over the cached rows (causal, aligned to the end), with log-sum-exp
  mass     the attention weight that every cached row received from the chunk, summed over rows and heads
  select   which cached rows stay when a cache is cut to a budget (first and latest positions, then most weight)
  move     moves the rows that stay beyond the budget into the freed places

Where `own` is false, `run` computes them with elementary torch operations in fp32; where it is true, with the
library's calls.  The lengths of a case are fixed by the case, the values by the seed.
"""
import math

import torch

own = False

D = 256  # head width of the full-context layers


# ----------------------------------------------------------------------------- cases


def listed():
    return [
        # two short conversations, one new token each: nothing but latency
        dict(name="attn_decode_small", op="attn", batch=2, q_long=1, n_long=0, kv_min=37, kv_max=321, heads=64,
             kv_heads=1, page=16, interleaved=False),
        # a serving batch in its decode phase, lengths spread from 1K to 32K, one pool for K and V
        dict(name="attn_decode_batch", op="attn", batch=32, q_long=1, n_long=0, kv_min=1024, kv_max=32768, heads=64,
             kv_heads=1, page=64, interleaved=True),
        # two prompts being read in odd chunks next to 22 decoding sequences, grouped heads
        dict(name="attn_mixed", op="attn", batch=24, q_long=389, n_long=2, kv_min=511, kv_max=8191, heads=32,
             kv_heads=4, page=32, interleaved=False),
        # a 2048-token chunk of a 32K prompt
        dict(name="attn_chunk_32k", op="attn", batch=1, q_long=2048, n_long=1, kv_min=32768, kv_max=32768, heads=64,
             kv_heads=1, page=64, interleaved=False),
        # the weights of a decode step over a serving batch
        dict(name="mass_decode_batch", op="mass", batch=32, q_long=1, n_long=0, kv_min=1024, kv_max=32768, heads=64,
             kv_heads=1, page=64, interleaved=False),
        # the weights of a prompt's chunk, odd lengths
        dict(name="mass_chunk_16k", op="mass", batch=1, q_long=1021, n_long=1, kv_min=16381, kv_max=16381, heads=64,
             kv_heads=1, page=64, interleaved=False),
        # a decode step's new rows
        dict(name="append_decode", op="append", batch=32, q_long=1, n_long=0, kv_min=1024, kv_max=8192, heads=64,
             kv_heads=1, page=64, interleaved=False),
        # the rows of two long prompt chunks, four K/V heads
        dict(name="append_chunk", op="append", batch=2, q_long=8192, n_long=2, kv_min=8192, kv_max=12345, heads=32,
             kv_heads=4, page=16, interleaved=True),
        # a cache kept near its budget: 128 rows over it in each of 32 sequences
        dict(name="select_steady", op="select", batch=32, kv=4224, budget=4096, n_sink=4, n_recent=256, kv_heads=1,
             page=64),
        # a long prompt cut to a quarter after it was read
        dict(name="select_long", op="select", batch=4, kv=131072, budget=32768, n_sink=16, n_recent=2048, kv_heads=1,
             page=64),
        # the steady state's moves
        dict(name="move_steady", op="move", batch=32, kv=4224, budget=4096, moves=121, kv_heads=1, page=64,
             interleaved=False),
        # the long prompt's moves
        dict(name="move_long", op="move", batch=4, kv=131072, budget=32768, moves=24571, kv_heads=1, page=64,
             interleaved=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "mass", "mass", "append", "select", "move"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op in ("attn", "mass", "append"):
        heads, kv_heads = rng.choice([(64, 1), (64, 1), (32, 4), (16, 1), (16, 16), (8, 2), (128, 1)])
        kind = rng.choice(["decode", "chunk", "mixed"])
        batch = {"decode": _log_int(rng, 1, 64), "chunk": rng.choice([1, 1, 2, 3]), "mixed": _log_int(rng, 4, 32)}[kind]
        q_long = 1 if kind == "decode" else _log_int(rng, 2, 2048)
        n_long = {"decode": 0, "chunk": batch, "mixed": max(1, batch // 8)}[kind]
        kv_max = _log_int(rng, max(16, q_long), 32768)
        # at most the rows and the products of the largest listed cases
        while batch * kv_max * kv_heads > 32 * 20000 or heads * (n_long * q_long + batch - n_long) * kv_max > 2.0e9:
            kv_max = kv_max * 3 // 4
            q_long = max(1, min(q_long, kv_max))
        kv_min = _log_int(rng, max(1, kv_max // 32), kv_max)
        return dict(op=op, batch=batch, q_long=q_long, n_long=n_long, kv_min=kv_min, kv_max=kv_max, heads=heads,
                    kv_heads=kv_heads, page=page, interleaved=rng.random() < 0.5)
    kv_heads = rng.choice([1, 1, 2, 8])
    batch = _log_int(rng, 1, 32)
    kv = _log_int(rng, 64, 131072)
    while batch * kv * kv_heads > 4 * 131072:
        kv = kv * 3 // 4
    budget = _log_int(rng, max(1, kv // 16), kv - 1)
    if op == "select":
        n_sink = rng.randint(0, min(16, budget))
        return dict(op=op, batch=batch, kv=kv, budget=budget, n_sink=n_sink,
                    n_recent=rng.randint(0, (budget - n_sink) // 2), kv_heads=kv_heads, page=page)
    return dict(op=op, batch=batch, kv=kv, budget=budget, moves=rng.randint(1, min(budget, kv - budget)),
                kv_heads=kv_heads, page=page, interleaved=rng.random() < 0.5)


def _lengths(c):
    """New tokens and cached rows (the new ones included) of every sequence."""
    if "kv" in c:
        return [0] * c["batch"], [c["kv"]] * c["batch"]
    q = [c["q_long"] if b < c["n_long"] else 1 for b in range(c["batch"])]
    share = [1.0 if b == 0 else (b * 0.6180339887) % 1.0 for b in range(c["batch"])]
    kv = [max(n, c["kv_min"] + int(s * (c["kv_max"] - c["kv_min"]))) for n, s in zip(q, share)]
    return q, kv


def work(case):
    c = case
    q, kv = _lengths(c)
    hk = c["kv_heads"]
    if c["op"] in ("attn", "mass"):
        h = c["heads"]
        pairs = sum(n * k - n * (n - 1) // 2 for n, k in zip(q, kv))  # (new token, cached row it sees)
        rows = sum(kv) * hk
        if c["op"] == "attn":
            return {"bytes": sum(q) * h * (2 * D * 2 + 4) + rows * 2 * D * 2, "flops": 4 * D * h * pairs}
        return {"bytes": sum(q) * h * (D * 2 + 4) + rows * (D * 2 + 4), "flops": 2 * D * h * pairs}
    if c["op"] == "append":
        return {"bytes": sum(q) * hk * (2 * 2 * D * 2 + 8), "flops": 0}
    if c["op"] == "select":
        n = c["batch"] * hk
        return {"bytes": n * (c["kv"] * 8 + min(c["budget"], _pages(c) * c["page"] - c["budget"]) * 8), "flops": 0}
    return {"bytes": c["batch"] * hk * c["moves"] * (2 * 2 * D * 2 + 16 + 8), "flops": 0}


def _pages(c):
    """Width of the page table."""
    return -(-max(_lengths(c)[1]) // c["page"])


# ----------------------------------------------------------------------------- inputs


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    q_len, kv_len = _lengths(c)
    B, hk, page, width = c["batch"], c["kv_heads"], c["page"], _pages(c)
    n_pages = B * width + 3
    s = dict(case=dict(c), q_len=q_len, kv=kv_len)
    s["cu_q"] = torch.tensor([0] + torch.tensor(q_len).cumsum(0).tolist(), dtype=torch.int32, device=dev)
    s["kv_len"] = torch.tensor(kv_len, dtype=torch.int32, device=dev)
    # the pages of a sequence lie anywhere in the pool
    s["table"] = torch.randperm(n_pages, generator=g, device=dev)[: B * width].reshape(B, width).to(torch.int32)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)

    if c["op"] != "select":
        if c["interleaved"]:
            pool = normal(n_pages, 2, page, hk, D)
            s["k_pool"], s["v_pool"] = pool[:, 0], pool[:, 1]
        else:
            s["k_pool"], s["v_pool"] = normal(n_pages, page, hk, D), normal(n_pages, page, hk, D)
    T = sum(q_len)
    if c["op"] in ("attn", "mass"):
        s["q"] = normal(T, c["heads"], D)
        if c["op"] == "mass":
            s["lse"] = _plain_attn(s, with_values=False)[1]
    elif c["op"] == "append":
        s["k"], s["v"] = normal(T, hk, D), normal(T, hk, D)
        s["seen"] = s["kv_len"] + torch.randint(0, 1000, (B,), generator=g, device=dev, dtype=torch.int32)
        s["pos"] = torch.randint(0, 100000, (n_pages, page, hk), generator=g, device=dev, dtype=torch.int32)
        s["mass"] = torch.rand((n_pages, page, hk), generator=g, device=dev)
    elif c["op"] == "select":
        n, budget, sink, recent = c["kv"], c["budget"], c["n_sink"], c["n_recent"]
        # positions: earlier evictions left gaps in the middle; rows moved into freed places are out of order
        gaps = torch.randint(1, 4, (B, n, hk), generator=g, device=dev)
        gaps[:, n - recent:] = 1
        seen = 4 * n + 32
        pos = seen - gaps.flip(1).cumsum(1).flip(1)
        pos[:, :sink] = torch.arange(sink, device=dev)[None, :, None]
        order = torch.rand((B, n, hk), generator=g, device=dev)
        order[:, budget:] = 2.0 + torch.arange(n - budget, device=dev)[None, :, None]
        pos = pos.gather(1, order.argsort(dim=1))
        # weights: heavy-tailed, and none yet for one row in ten
        mass = torch.exp(2.0 * torch.randn((B, n, hk), generator=g, device=dev))
        mass = torch.where(torch.rand((B, n, hk), generator=g, device=dev) < 0.1, torch.zeros_like(mass), mass)
        s["seen"] = torch.full((B,), seen, dtype=torch.int32, device=dev)
        s["pos"] = torch.zeros((n_pages, page, hk), dtype=torch.int32, device=dev)
        s["mass"] = torch.zeros((n_pages, page, hk), device=dev)
        slot = _slots(s)
        s["pos"].view(-1, hk)[slot] = pos.to(torch.int32)
        s["mass"].view(-1, hk)[slot] = mass
    else:
        n, budget, m = c["kv"], c["budget"], c["moves"]
        limit = min(budget, width * page - budget)
        dst = torch.rand((B, hk, budget), generator=g, device=dev).topk(m, dim=2).indices.sort(dim=2).values
        src = torch.rand((B, hk, n - budget), generator=g, device=dev).topk(m, dim=2).indices.sort(dim=2).values
        s["moves"] = torch.full((B, hk, limit, 2), -1, dtype=torch.int32, device=dev)
        s["moves"][:, :, :m, 0] = (src + budget).to(torch.int32)
        s["moves"][:, :, :m, 1] = dst.to(torch.int32)
        s["pos"] = torch.randint(0, 100000, (n_pages, page, hk), generator=g, device=dev, dtype=torch.int32)
        s["mass"] = torch.rand((n_pages, page, hk), generator=g, device=dev)
    return s


def _slots(s):
    """Pool row (page * page size + offset) of every row of every sequence, [B, longest]."""
    page = s["case"]["page"]
    i = torch.arange(max(s["kv"]), device="cuda")
    return s["table"][:, i // page].long() * page + i % page


# ----------------------------------------------------------------------------- plain forms


def _rows(pool, slot):
    """Rows of a pool [pages, page, heads, ...] (its first stride may be larger) by pool row number."""
    page = pool.shape[1]
    return pool[slot // page, slot % page]


def _plain_group(q, k, v, first):
    """q [N, n, heads, D], k, v [N, L, kv heads, D]; query i of batch entry b sees the rows <= first[b] + i.
    Returns the output and the log-sum-exp in fp32."""
    N, n, H, _ = q.shape
    L, hk = k.shape[1], k.shape[2]
    g = H // hk
    qf = q.float().reshape(N, n, hk, g, D).permute(0, 2, 1, 3, 4).reshape(N, hk, n * g, D)
    x = (qf @ k.float().permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(D)).view(N, hk, n, g, L)
    hidden = torch.arange(L, device=q.device) > first[:, None, None] + torch.arange(n, device=q.device)[:, None]
    x.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True).clamp_min(-3.0e38)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0].permute(0, 2, 1, 3).reshape(N, n, H)
    if v is None:
        return None, lse
    o = x.view(N, hk, n * g, L) @ v.float().permute(0, 2, 1, 3) / total.view(N, hk, n * g, 1)
    return o.view(N, hk, n, g, D).permute(0, 2, 1, 3, 4).reshape(N, n, H, D), lse


def _plain_attn(s, with_values=True):
    slot, q = _slots(s), s["q"]
    if max(s["q_len"]) == 1:  # one new token each: one padded batch
        v = _rows(s["v_pool"], slot) if with_values else None
        o, lse = _plain_group(q[:, None], _rows(s["k_pool"], slot), v, s["kv_len"] - 1)
        return (o[:, 0].to(q.dtype) if with_values else None), lse[:, 0]
    outs, lses, t = [], [], 0
    for b, (n, kv) in enumerate(zip(s["q_len"], s["kv"])):  # a ragged batch: each sequence at its own lengths
        rows = slot[b : b + 1, :kv]
        v = _rows(s["v_pool"], rows) if with_values else None
        o, lse = _plain_group(q[None, t : t + n], _rows(s["k_pool"], rows), v, s["kv_len"][b : b + 1] - n)
        outs.append(o[0].to(q.dtype) if with_values else None)
        lses.append(lse[0])
        t += n
    return (torch.cat(outs) if with_values else None), torch.cat(lses)


def _plain_weights(q, k, lse, first):
    """Sum over queries and heads of exp(score - lse): [N, L, kv heads]."""
    N, n, H, _ = q.shape
    L, hk = k.shape[1], k.shape[2]
    g = H // hk
    qf = q.float().reshape(N, n, hk, g, D).permute(0, 2, 1, 3, 4).reshape(N, hk, n * g, D)
    x = (qf @ k.float().permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(D)).view(N, hk, n, g, L)
    x.sub_(lse.reshape(N, n, hk, g).permute(0, 2, 1, 3)[..., None]).exp_()
    hidden = torch.arange(L, device=q.device) > first[:, None, None] + torch.arange(n, device=q.device)[:, None]
    x.masked_fill_(hidden[:, None, :, None, :], 0.0)
    return x.sum((2, 3)).transpose(1, 2)


def _plain_mass(s):
    slot, q, hk = _slots(s), s["q"], s["case"]["kv_heads"]
    out = torch.zeros(s["k_pool"].shape[:3], device="cuda")
    flat = out.view(-1, hk)
    if max(s["q_len"]) == 1:
        w = _plain_weights(q[:, None], _rows(s["k_pool"], slot), s["lse"][:, None], s["kv_len"] - 1)
        flat.index_add_(0, slot.reshape(-1), w.reshape(-1, hk))
        return out
    t = 0
    for b, (n, kv) in enumerate(zip(s["q_len"], s["kv"])):
        rows = slot[b : b + 1, :kv]
        w = _plain_weights(q[None, t : t + n], _rows(s["k_pool"], rows), s["lse"][None, t : t + n],
                           s["kv_len"][b : b + 1] - n)
        flat.index_add_(0, rows[0], w[0])
        t += n
    return out


def _plain_append(s):
    cu, page = s["cu_q"].long(), s["case"]["page"]
    t = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    back = cu[b + 1] - t  # rows from here to the end of the sequence
    i = s["kv_len"].long()[b] - back
    p, r = s["table"][b, i // page].long(), i % page
    s["k_pool"][p, r] = s["k"]
    s["v_pool"][p, r] = s["v"]
    s["pos"][p, r] = (s["seen"].long()[b] - back).to(torch.int32)[:, None]
    s["mass"][p, r] = 0.0


def _plain_select(s):
    c = s["case"]
    n, budget, hk, B = c["kv"], c["budget"], c["kv_heads"], c["batch"]
    slot = _slots(s)
    pos = s["pos"].view(-1, hk)[slot].transpose(1, 2)  # [B, heads, n]
    mass = s["mass"].view(-1, hk)[slot].transpose(1, 2)
    seen = s["seen"][:, None, None]
    safe = (pos < c["n_sink"]) | (pos >= seen - c["n_recent"])
    order = torch.where(safe, torch.full_like(mass, math.inf), mass).argsort(dim=2, descending=True, stable=True)
    keep = torch.zeros((B, hk, n), dtype=torch.bool, device="cuda").scatter_(2, order[:, :, :budget], True)
    free, late = ~keep[:, :, :budget], keep[:, :, budget:]
    limit = min(budget, s["table"].shape[1] * c["page"] - budget)
    moves = torch.full((B, hk, limit, 2), -1, dtype=torch.int32, device="cuda")
    for side, there, at in ((0, late, budget), (1, free, 0)):
        where = there.nonzero()
        rank = (there.cumsum(2) - 1)[there]
        moves[where[:, 0], where[:, 1], rank, side] = (where[:, 2] + at).to(torch.int32)
    return moves, s["kv_len"].clamp_max(budget)


def _plain_move(s):
    c, table, moves = s["case"], s["table"].long(), s["moves"].long()
    page = c["page"]
    b, h, i = (moves[..., 0] >= 0).nonzero(as_tuple=True)
    src, dst = moves[b, h, i, 0], moves[b, h, i, 1]
    ps, rs, pd, rd = table[b, src // page], src % page, table[b, dst // page], dst % page
    for name in ("k_pool", "v_pool", "pos", "mass"):
        s[name][pd, rd, h] = s[name][ps, rs, h]


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import sparse_attention_hca_b200 as hd

        if op == "attn":
            return hd.mla_paged_attn_fwd(s["q"], s["k_pool"], s["v_pool"], s["table"], s["cu_q"], s["kv_len"],
                                         return_lse=True)
        if op == "mass":
            return hd.mla_paged_attn_mass(s["q"], s["k_pool"], s["table"], s["cu_q"], s["kv_len"], s["lse"])
        if op == "append":
            hd.mla_cache_append(s["k"], s["v"], s["k_pool"], s["v_pool"], s["table"], s["cu_q"], s["kv_len"],
                                seen=s["seen"], pos=s["pos"], mass=s["mass"])
        elif op == "select":
            c = s["case"]
            return hd.mla_evict_select(s["mass"], s["pos"], s["table"], s["kv_len"], s["seen"], c["budget"],
                                       n_sink=c["n_sink"], n_recent=c["n_recent"])
        else:
            hd.mla_cache_move(s["moves"], s["k_pool"], s["v_pool"], s["table"], pos=s["pos"], mass=s["mass"])
        return s["k_pool"], s["v_pool"], s["pos"], s["mass"]
    if op == "attn":
        return _plain_attn(s)
    if op == "mass":
        return _plain_mass(s)
    if op == "select":
        return _plain_select(s)
    (_plain_append if op == "append" else _plain_move)(s)
    return s["k_pool"], s["v_pool"], s["pos"], s["mass"]


# ----------------------------------------------------------------------------- from the definitions, in 64 bits


def exact(case, seed):
    s, c = prepare(case, seed), case
    op, page, hk = c["op"], c["page"], c["kv_heads"]
    if op == "select":
        return None
    table = s["table"].long()
    if op in ("append", "move"):
        k, v, m = (s[n].double() for n in ("k_pool", "v_pool", "mass"))
        if op == "append":
            t = 0
            for b, (n, kv) in enumerate(zip(s["q_len"], s["kv"])):
                at = torch.arange(kv - n, kv, device="cuda")
                to = (table[b, torch.div(at, page, rounding_mode="floor")], at.remainder(page))
                k[to], v[to], m[to] = s["k"][t : t + n].double(), s["v"][t : t + n].double(), 0.0
                t += n
        else:
            for b in range(c["batch"]):
                for h in range(hk):
                    a, z = s["moves"][b, h, : c["moves"]].long().unbind(1)
                    here = (table[b, torch.div(a, page, rounding_mode="floor")], a.remainder(page))
                    to = (table[b, torch.div(z, page, rounding_mode="floor")], z.remainder(page))
                    for x in (k, v, m):
                        x[:, :, h][to] = x[:, :, h][here]
        return k, v, None, m
    H = c["heads"]
    group = H // hk
    outs, lses, t = [], [], 0
    mass = torch.zeros(s["k_pool"].shape[:3], dtype=torch.float64, device="cuda")
    for b, (n, kv) in enumerate(zip(s["q_len"], s["kv"])):
        at = torch.arange(kv, device="cuda")
        there = (table[b, torch.div(at, page, rounding_mode="floor")], at.remainder(page))
        k = s["k_pool"][there].double()
        v = s["v_pool"][there].double()
        o = torch.empty((n, H, D), dtype=torch.float64, device="cuda")
        e = torch.empty((n, H), dtype=torch.float64, device="cuda")
        w = torch.zeros((kv, hk), dtype=torch.float64, device="cuda")
        for i0 in range(0, n, 256):
            i1 = min(n, i0 + 256)
            seen = at[None] <= torch.arange(kv - n + i0, kv - n + i1, device="cuda")[:, None]
            for h in range(H):
                x = s["q"][t + i0 : t + i1, h].double() @ k[:, h // group].T / 16.0
                x = torch.where(seen, x, -math.inf)
                if op == "attn":
                    e[i0:i1, h] = torch.logsumexp(x, 1)
                    o[i0:i1, h] = torch.softmax(x, 1) @ v[:, h // group]
                else:
                    w[:, h // group] += torch.exp(x - s["lse"][t + i0 : t + i1, h, None].double()).sum(0)
        outs.append(o)
        lses.append(e)
        mass[there] += w
        t += n
    return (torch.cat(outs), torch.cat(lses)) if op == "attn" else mass
