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
