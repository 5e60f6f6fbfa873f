"""Refusals of the paged-cache calls of the full-context (MLA) layers, without a GPU: the C entry
points return their status before touching device memory, and the Python binding rejects tensors
that do not fit together."""
import pytest
import torch

import sparse_attention_hca_b200 as hd

F = 1 << 20  # never dereferenced: every call below fails its checks first, or has nothing to do
bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_hca_b200 import build

    build.build()
    return hd.lib()


APPEND = dict(K=F, V=F, kr=256, vr=256, Kp=F, Vp=F, kp=16384, vp=16384, table=F, cu=F, kv=F, seen=None, pos=None,
              mass=None, B=2, T=4, n_pages=8, page=64, max_pages=3, Hkv=1, d=256, s=None)
ATTN = dict(Q=F, qr=16384, Kp=F, Vp=F, kp=16384, vp=16384, table=F, cu=F, kv=F, O=F, lse=None, B=2, T=4, n_pages=8,
            page=64, max_pages=3, Hq=64, Hkv=1, d=256, scale=0.0625, ws=None, wsb=0, s=None)
MASS = dict(Q=F, qr=16384, Kp=F, kp=16384, table=F, cu=F, kv=F, lse=F, mass=F, B=2, T=4, n_pages=8, page=64,
            max_pages=3, Hq=64, Hkv=1, d=256, scale=0.0625, ws=None, wsb=0, s=None)
SELECT = dict(mass=F, pos=F, table=F, kv=F, seen=None, moves=F, new=F, B=2, n_pages=8, page=64, max_pages=3, Hkv=1,
              budget=100, n_sink=4, n_recent=50, n_moves=92, s=None)
MOVE = dict(moves=F, table=F, Kp=F, Vp=F, kp=16384, vp=16384, pos=None, mass=None, B=2, n_moves=5, n_pages=8, page=64,
            max_pages=3, Hkv=1, d=256, s=None)
CALLS = dict(mla_cache_append=APPEND, mla_paged_attn_fwd=ATTN, mla_paged_attn_mass=MASS, mla_evict_select=SELECT,
             mla_cache_move=MOVE)


@pytest.mark.parametrize("name", list(CALLS))
def test_common_refusals(lib, name):
    args = CALLS[name]

    def call(**kw):
        return getattr(lib, name)(*dict(args, **kw).values())

    for k, v in args.items():
        if v == F:
            assert call(**{k: None}) == -1, k
    for k in ("table", "cu", "kv"):
        if k in args:
            assert call(**{k: F + 2}) == -3, k
    for k in ("K", "V", "Q", "Kp", "Vp", "O"):
        if k in args:
            assert call(**{k: F + 8}) == -3, k
    assert call(page=48, kp=1 << 20, vp=1 << 20) == -4 if "kp" in args and "vp" in args else call(page=48) == -4
    assert call(page=8) == -4
    assert call(n_pages=0) == -2 and call(max_pages=0) == -2 and call(B=-1) == -2 and call(Hkv=0) == -2
    if "kp" in args:
        assert call(kp=16383) == -2
        assert call(kp=16388) == -3
    if "d" in args:
        assert call(d=128) == -4
    assert call(B=0) == 0


def test_query_refusals(lib):
    for name in ("mla_paged_attn_fwd", "mla_paged_attn_mass"):
        def call(**kw):
            return getattr(lib, name)(*dict(CALLS[name], **kw).values())

        assert call(Hq=48, qr=48 * 256) == -4           # 48 heads per K/V head
        assert call(Hq=256, qr=256 * 256) == -4
        assert call(Hq=7, Hkv=2, kp=1 << 20) == -2
        assert call(qr=16383) == -2 and call(qr=16388) == -3
        assert call(scale=0.0) == -2 and call(scale=-1.0) == -2 and call(scale=float("nan")) == -2
        assert call(T=-1) == -2 and call(T=0) == 0
        assert call(T=(1 << 23) + 1) == -4
    for bad in ((-1, 4, 64, 1), (2, 4, 48, 1), (2, 4, 7, 2), (0, 4, 64, 1), (2, 0, 64, 1), (2, 4, 0, 1), (2, 4, 64, 0)):
        assert lib.mla_paged_attn_fwd_workspace_size(*bad) == 0
        assert lib.mla_paged_attn_mass_workspace_size(*bad) == 0


def test_select_refusals(lib):
    def call(**kw):
        return lib.mla_evict_select(*dict(SELECT, **kw).values())

    assert call(budget=0) == -2 and call(n_sink=-1) == -2 and call(n_recent=-1) == -2
    assert call(n_recent=97) == -2                       # protected rows beyond the budget
    assert call(n_moves=91) == -2                        # 192 rows cut to 100: 92 moves
    assert call(moves=F + 4) == -3


def _tensors(B=2, T=4, Hq=64, Hkv=1, page=64, n_pages=8, width=3):
    t = dict(q=torch.zeros(T, Hq, 256, dtype=bf), k=torch.zeros(T, Hkv, 256, dtype=bf),
             K=torch.zeros(n_pages, page, Hkv, 256, dtype=bf), V=torch.zeros(n_pages, page, Hkv, 256, dtype=bf),
             table=torch.zeros(B, width, dtype=i32), cu=torch.zeros(B + 1, dtype=i32), kv=torch.zeros(B, dtype=i32),
             lse=torch.zeros(T, Hq), mass=torch.zeros(n_pages, page, Hkv), pos=torch.zeros(n_pages, page, Hkv, dtype=i32),
             moves=torch.zeros(B, Hkv, 5, 2, dtype=i32))
    return t


@pytest.mark.parametrize("what,how", [
    ("V", lambda t: t["V"][:4]), ("K", lambda t: t["K"].float()), ("K", lambda t: t["K"].transpose(1, 2)),
    ("K", lambda t: t["K"][:, ::2]), ("table", lambda t: t["table"].long()), ("table", lambda t: t["table"][0]),
    ("table", lambda t: t["table"][:, :2]), ("cu", lambda t: t["cu"][:2]), ("kv", lambda t: t["kv"][:1]),
    ("q", lambda t: t["q"][..., :128].contiguous()), ("q", lambda t: t["q"].transpose(0, 1)),
    ("q", lambda t: t["q"][0]), ("q", lambda t: t["q"].half())])
def test_attention_rejects_mismatched_tensors(what, how):
    t = _tensors()
    t[what] = how(t)
    with pytest.raises(ValueError, match=r"shape|must be"):
        hd.mla_paged_attn_fwd(t["q"], t["K"], t["V"], t["table"], t["cu"], t["kv"])
    if what != "V":
        with pytest.raises(ValueError, match=r"shape|must be"):
            hd.mla_paged_attn_mass(t["q"], t["K"], t["table"], t["cu"], t["kv"], t["lse"])


def test_outputs_and_side_inputs_are_checked():
    t = _tensors()
    a = (t["q"], t["K"], t["V"], t["table"], t["cu"], t["kv"])
    for kw in (dict(O=torch.zeros(3, 64, 256, dtype=bf)), dict(lse=torch.zeros(4, 1)), dict(O=torch.zeros(4, 64, 256))):
        with pytest.raises(ValueError):
            hd.mla_paged_attn_fwd(*a, **kw)
    with pytest.raises(ValueError, match="lse"):
        hd.mla_paged_attn_mass(t["q"], t["K"], t["table"], t["cu"], t["kv"], t["lse"][:3])
    with pytest.raises(ValueError, match="mass"):
        hd.mla_paged_attn_mass(t["q"], t["K"], t["table"], t["cu"], t["kv"], t["lse"], mass=t["mass"][:2])
    for kw in (dict(pos=t["pos"][:1]), dict(mass=t["mass"].double()), dict(seen=t["kv"][:1])):
        with pytest.raises(ValueError):
            hd.mla_cache_append(t["k"], t["k"], t["K"], t["V"], t["table"], t["cu"], t["kv"], **kw)
    with pytest.raises(ValueError):
        hd.mla_cache_append(t["k"], t["k"][:3], t["K"], t["V"], t["table"], t["cu"], t["kv"])
    with pytest.raises(ValueError, match="new_len must not be kv_len"):
        hd.mla_evict_select(t["mass"], t["pos"], t["table"], t["kv"], None, 100, new_len=t["kv"])
    with pytest.raises(ValueError, match="pos"):
        hd.mla_evict_select(t["mass"], t["pos"][:1], t["table"], t["kv"], None, 100)
    with pytest.raises(ValueError, match="moves"):
        hd.mla_cache_move(t["moves"][:1], t["K"], t["V"], t["table"])
    # everything fits, but nothing lies on a GPU
    for call in (lambda: hd.mla_paged_attn_fwd(*a), lambda: hd.mla_cache_move(t["moves"], t["K"], t["V"], t["table"]),
                 lambda: hd.mla_evict_select(t["mass"], t["pos"], t["table"], t["kv"], None, 100)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
