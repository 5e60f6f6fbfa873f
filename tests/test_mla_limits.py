"""Further refusals of the paged-cache calls of the full-context (MLA) layers, without a GPU."""
import os

import pytest
import torch
from test_mla_checks import F, SELECT, _tensors, i32, lib  # noqa: F401  (lib: a fixture)

import sparse_attention_hca_b200 as hd


@pytest.mark.parametrize("kw", [dict(n_recent=2 ** 32), dict(n_sink=2 ** 32), dict(n_recent=2 ** 31), dict(n_sink=-(2 ** 32)),
                                dict(n_recent=-(2 ** 31) - 1), dict(budget=2 ** 32 + 100), dict(budget=-(2 ** 32) + 100),
                                dict(budget=2 ** 64 + 100)])
def test_select_counts_beyond_32_bits(kw):
    """Counts are C ints: one that does not fit is refused, not taken modulo 2^32."""
    t = _tensors()
    kw = dict(dict(budget=100, n_sink=4, n_recent=50), **kw)
    with pytest.raises(ValueError, match="32-bit"):
        hd.mla_evict_select(t["mass"], t["pos"], t["table"], t["kv"], None, kw.pop("budget"), **kw)


def test_sizes_beyond_32_bits():
    """Nor do sizes of tensors wrap: a table or a list of moves as wide as 2^32, or as many sequences."""
    t = _tensors()
    wide = torch.empty(2, 2 ** 32 + 3, dtype=i32, device="meta")
    with pytest.raises(ValueError, match="32-bit"):
        hd.mla_paged_attn_fwd(t["q"], t["K"], t["V"], wide, t["cu"], t["kv"])
    with pytest.raises(ValueError, match="32-bit"):
        hd.mla_paged_attn_mass(t["q"], t["K"], torch.empty(2 ** 32 + 2, 3, dtype=i32, device="meta"), t["cu"], t["kv"],
                               t["lse"])
    with pytest.raises(ValueError, match="32-bit"):
        hd.mla_evict_select(t["mass"], t["pos"], wide, t["kv"], None, 100)
    with pytest.raises(ValueError, match="32-bit"):
        hd.mla_cache_move(t["moves"], t["K"], t["V"], wide)
    with pytest.raises(ValueError, match="32-bit"):
        hd.mla_cache_move(torch.empty(2, 1, 2 ** 32 + 5, 2, dtype=i32, device="meta"), t["K"], t["V"], t["table"])


def test_select_lengths_may_not_overlap():
    """new_len is written while other lists still read kv_len and seen."""
    t = _tensors(B=3)
    buf = torch.zeros(8, dtype=i32)
    for kv, seen, new in ((buf[0:3], None, buf[0:3]), (buf[0:3], None, buf[2:5]), (buf[2:5], None, buf[0:3]),
                          (buf[0:3], buf[3:6], buf[3:6]), (buf[0:3], buf[3:6], buf[5:8])):
        with pytest.raises(ValueError, match="new_len must not"):
            hd.mla_evict_select(t["mass"], t["pos"], t["table"], kv, seen, 100, new_len=new)
    with pytest.raises(ValueError, match="CUDA"):  # side by side is fine; nothing lies on a GPU
        hd.mla_evict_select(t["mass"], t["pos"], t["table"], buf[0:3], None, 100, new_len=buf[3:6])


def test_select_lengths_may_not_overlap_in_c(lib):  # noqa: F811
    def call(**kw):
        return lib.mla_evict_select(*dict(SELECT, moves=2 * F, **kw).values())

    assert call(kv=F, new=F) == -2 and call(kv=F, new=F + 4) == -2 and call(kv=F + 4, new=F) == -2
    assert call(kv=F, seen=F + 64, new=F + 64) == -2 and call(kv=F, seen=F + 64, new=F + 68) == -2
    assert call(kv=F, seen=F, new=F + 8, B=0) == 0


@pytest.mark.parametrize("name", ["attn", "mass"])
def test_no_way_out_before_the_records(name):
    """The merging kernel that follows trusts every worker's record in the workspace, so the main kernel may not end
    before it has written its own."""
    with open(os.path.join(os.path.dirname(hd.__file__), "csrc", f"mla_{name}.cu")) as f:
        text = f.read()
    body = text[text.index(f"{name}_kernel(const __grid_constant__") :]
    body = body[: body.index("launch_dependents();")]
    assert "p.ws_meta + worker * kMetaInts" in body
    assert "return;" not in body
