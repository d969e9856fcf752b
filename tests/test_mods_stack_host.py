"""What AttnStack holds and hands to the calls with modified scores, on the host: calls that launch are replaced by ones
that note their arguments (no GPU needed)."""

import pytest
import torch

from gemma_dual_geometry_gb300 import build as g4build
from gemma_dual_geometry_gb300 import g4attn as G
from gemma_dual_geometry_gb300 import stack as S
from gemma_dual_geometry_gb300 import workloads as W

CFG = dict(B=70, H=4, Hkv=2, dtype=W.BF16, seed=0, types=[W.SLIDING, W.FULL, W.SLIDING, W.FULL], n_shared=2,
           geom={W.SLIDING: dict(head_dim=64, theta=1e4, rotary_fraction=1.0, window=700),
                 W.FULL: dict(head_dim=128, theta=1e6, rotary_fraction=0.25, window=0)})


@pytest.fixture
def calls(monkeypatch):
    """(name, arguments by position) of the calls made."""
    g4build.build()
    G.lib()
    seen = []
    for name in ("g4_attn_visible_ranges", "g4_kv_append_normrope_axes", "g4_attn_decode_mods"):
        monkeypatch.setattr(G, name, lambda *a, stream=None, name=name: seen.append((name, a)))
    return seen


def make(cfg=CFG, **kw):
    return S.AttnStack(cfg, 800, device="cpu", **kw)


def test_a_workspace_for_each_layer(calls):
    """As for the plain decodes: layers' decodes may run at the same time (the stack had one for all)."""
    st = make(mods=True)
    mods = G.score_mods(30.0)
    for l in range(st.n):
        st.decode_attn(l, None, None, 800, None, mods=mods)
    spaces = [a[9] for _, a in calls]
    assert len({ws.data_ptr() for ws in spaces}) == st.n
    for l, (_, a) in enumerate(calls):
        need = G.g4_attn_decode_mods_workspace_size(st.params[l], 70, 800)
        assert need > 0 and a[10] >= need and a[9].numel() == a[10] and not a[9].any()
    with pytest.raises(ValueError, match="without mods"):
        make().decode_attn(0, None, None, 800, None, mods=mods)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_intervals_of_a_layer_type(calls):
    """Each type's window; types that no layer has, and arrays of other types or sizes, are refused (ids of T columns were
    read past their end)."""
    st = make()
    B, T, L = 70, 5, 800
    good = [i32(B), i32(B), i32(B, L), i32(B, L), T, i32(B, T), i32(B, T)]
    for lt, window in ((W.SLIDING, 700), (W.FULL, 0)):
        st.visible_ranges(lt, *good)
        assert calls[-1][1][:2] == (window, good[0]) and calls[-1][1][5:8] == (L, B, T)
    st.visible_ranges(W.FULL, 4096, good[1], None, None, T, *good[5:])   # (addresses; no ids)
    st.visible_ranges(W.FULL, *good[:5], i32(B * T + 9), i32(B * T))     # (flat buffers, longer than that)
    n = len(calls)
    for at, bad in ((0, i32(B - 1)), (0, i32(B).long()), (1, i32(B, 2)), (2, i32(B, T)), (3, i32(B, L).float()),
                    (3, i32(L, B).t()), (2, i32(1, L)), (5, i32(B, T + 1)), (6, i32(B)), (6, i32(B * T - 1)), (5, i32(B, T).long())):
        with pytest.raises(ValueError, match="int32"):
            st.visible_ranges(W.FULL, *good[:at], bad, *good[at + 1:])
    full_only = S.AttnStack(dict(CFG, types=[W.FULL, W.FULL], n_shared=0), 800, device="cpu")
    for lt in (W.SLIDING, 7):
        with pytest.raises(ValueError, match="no layers"):
            full_only.visible_ranges(lt, *good)
    assert len(calls) == n


def test_positions_and_rows_of_an_append(calls):
    st = make()
    B, T = 70, 4
    for l in range(4):
        axes = G.rope_axes(3, [0] * 64, 128)
        pos, rows = i32(3, B, T), i32(B, T)
        st.append_axes(l, axes, None, None, None, None, None, pos, rows, T, None)
        assert calls[-1][1][9] is pos and (calls[-1][1][10] is rows) == st.owns(l)
        n = len(calls)
        for p, r in ((i32(B, T), rows), (pos.long(), rows), (i32(3, T, B).transpose(1, 2), rows), (pos, i32(B, T + 1)),
                     (pos, rows.long())):
            if p is not pos or st.owns(l):
                with pytest.raises(ValueError, match="int32"):
                    st.append_axes(l, axes, None, None, None, None, None, p, r, T, None)
        assert len(calls) == n
