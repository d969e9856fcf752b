"""Refusals of the calls with modified scores, intervals and several axes (no GPU needed: every call here is refused
before a launch, or has nothing to launch)."""

import pytest
import torch

from gemma_dual_geometry_gb300 import build as g4build
from gemma_dual_geometry_gb300 import g4attn as G

FAKE = 0x7f0000000000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    g4build.build()
    return G.lib()


def params(**kw):
    d = dict(layer_type=G.G4_SLIDING, head_dim=256, n_heads=8, n_kv_heads=2, window=512, dtype=G.G4_BF16)
    d.update(kw)
    return G.layer_params(**d)


def table(max_len=100, batch=2, ring=False, dtype=G.G4_BF16, layer_type=G.G4_SLIDING, head_dim=256):
    t = G.cache_table(2)
    G.set_cache(t, 0, FAKE, FAKE + 4096, layer_type, head_dim, 2, max_len, batch, dtype, ring)
    return t


def status(fn, *args, **kw):
    try:
        fn(*args, **kw)
        return G.G4_OK
    except G.G4Error as e:
        return e.status


def test_visible_ranges(L):
    def call(window=0, start=FAKE, lens=FAKE, doc=FAKE, span=FAKE, max_len=10, B=1, T=0, begin=FAKE, end=FAKE):
        return status(G.g4_attn_visible_ranges, window, start, lens, doc, span, max_len, B, T, begin, end, 0)

    assert call() == G.G4_OK and call(B=0, T=5) == G.G4_OK and call(doc=None, span=None) == G.G4_OK
    assert call(max_len=1 << 24) == G.G4_OK
    for kw in (dict(window=-1), dict(B=-1), dict(T=-1), dict(max_len=0), dict(start=None), dict(lens=None),
               dict(begin=None), dict(end=None), dict(B=1 << 15, T=1 << 16)):
        assert call(**kw) == G.G4_ERR_INVALID_ARG, kw
    assert call(max_len=(1 << 24) + 1) == G.G4_ERR_UNSUPPORTED
    assert call(B=(1 << 20) + 1) == G.G4_ERR_UNSUPPORTED


def test_append_axes(L):
    axes = G.rope_axes(3, [0] * 40 + [1] * 40 + [2] * 48, 256)

    def call(p=None, t=None, axes=axes, layer=0, q=FAKE, k=FAKE, v=FAKE, qw=FAKE, kw=FAKE, pos=FAKE, rows=FAKE, B=2, T=0,
             out=FAKE):
        return status(G.g4_kv_append_normrope_axes, p or params(), t or table(1000), layer, axes, q, k, v, qw, kw, pos,
                      rows, B, T, out, 0)

    assert call() == G.G4_OK and call(B=0, T=4) == G.G4_OK
    shared = dict(p=params(kv_share_src=0), layer=1, k=None, v=None, kw=None, rows=None)
    assert call(**shared) == G.G4_OK
    for kw in (dict(B=-1), dict(T=-1), dict(q=None), dict(k=None), dict(v=None), dict(kw=None), dict(rows=None),
               dict(pos=None), dict(out=None), dict(out=FAKE + 8), dict(q=FAKE + 8), dict(qw=FAKE + 4), dict(layer=2),
               dict(shared, k=FAKE), dict(shared, layer=5),
               dict(axes=G.rope_axes(2, [0] * 40 + [2] * 88, 256)),                  # an axis that there is not
               dict(axes=G.rope_axes(1, [0] * 128, 256, [1.5] + [0.1] * 127)),       # a frequency above 1
               dict(axes=G.rope_axes(1, [0] * 128, 256, [-0.5] + [0.1] * 127)),
               dict(axes=G.rope_axes(1, [0] * 128, 256, [float("nan")] + [0.1] * 127))):
        assert call(**kw) == G.G4_ERR_INVALID_ARG, kw
    assert call(axes=G.rope_axes(0, [0] * 128, 256)) == G.G4_ERR_UNSUPPORTED
    assert call(axes=G.rope_axes(5, [0] * 128, 256)) == G.G4_ERR_UNSUPPORTED
    assert call(B=3) == G.G4_ERR_CAPACITY
    assert call(p=params(head_dim=128)) == G.G4_ERR_SHARE_MISMATCH
    assert call(t=table(511, ring=True)) == G.G4_ERR_CAPACITY
    # pairs that do not rotate may name any axis
    assert call(p=params(rotary_fraction=0.25), axes=G.rope_axes(1, [0] * 32 + [9] * 96, 256)) == G.G4_OK
    assert L.g4_kv_append_normrope_axes(params(), table(1000), 2, 0, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, 0,
                                        FAKE, None) == G.G4_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        G.rope_axes(1, [0] * 129, 256)
    with pytest.raises(ValueError):
        G.rope_axes(1, [0] * 128, 256, [0.5] * 129)


MODS = [(dict(softcap=2.0 ** -11), G.G4_ERR_UNSUPPORTED), (dict(softcap=1025.0), G.G4_ERR_UNSUPPORTED),
        (dict(softcap=-1.0), G.G4_ERR_UNSUPPORTED), (dict(softcap=float("nan")), G.G4_ERR_UNSUPPORTED),
        (dict(softcap=float("inf")), G.G4_ERR_UNSUPPORTED), (dict(slopes=FAKE + 2), G.G4_ERR_INVALID_ARG),
        (dict(key_begin=FAKE + 1), G.G4_ERR_INVALID_ARG),
        (dict(softcap=50.0, slopes=FAKE, key_begin=FAKE), G.G4_OK), (dict(softcap=2.0 ** -10), G.G4_OK)]


def test_prefill_mods(L):
    def call(p=None, t=None, mods=None, q=FAKE, start=FAKE, B=2, T=0, out=FAKE, layer=0):
        return status(G.g4_attn_prefill_mods, p or params(), t or table(), layer, mods, q, start, B, T, out, 0)

    for kw, want in MODS:
        assert call(mods=G.score_mods(**kw)) == want, kw
    assert call(mods=G.score_mods(key_begin=FAKE, key_end=FAKE)) == G.G4_OK
    assert call(mods=G.score_mods(key_end=FAKE + 2)) == G.G4_ERR_INVALID_ARG
    assert call() == G.G4_OK and call(B=0, T=4) == G.G4_OK
    for kw in (dict(q=None), dict(start=None), dict(out=None), dict(out=FAKE + 8), dict(B=-1), dict(T=-1), dict(layer=2)):
        assert call(**kw) == G.G4_ERR_INVALID_ARG, kw
    assert call(B=3) == G.G4_ERR_CAPACITY and call(T=101) == G.G4_ERR_CAPACITY
    assert call(p=params(head_dim=512)) == G.G4_ERR_SHARE_MISMATCH
    assert call(p=params(attn_scale=1e38), mods=G.score_mods(softcap=0.01)) == G.G4_ERR_UNSUPPORTED
    # rings: as in g4_attn_prefill, but intervals of the caller's own need no room for windows
    ring = table(1024, ring=True)
    assert call(t=ring, B=0, T=513) == G.G4_OK and call(t=ring, T=514) == G.G4_ERR_CAPACITY
    own = G.score_mods(key_begin=FAKE)
    assert call(t=ring, mods=own, B=0, T=1024) == G.G4_OK and call(t=ring, mods=own, T=1025) == G.G4_ERR_CAPACITY
    assert call(t=table(1000, ring=True), B=0, T=4) == G.G4_ERR_UNSUPPORTED


def test_decode_mods(L):
    need = G.g4_attn_decode_mods_workspace_size(params(), 64, 8192)
    assert need > 0 and need % 256 == 0
    assert G.g4_attn_decode_mods_workspace_size(params(), 0, 8192) == 0
    assert L.g4_attn_decode_mods_workspace_size(None, 64, 8192) == 0

    def call(p=None, t=None, mods=None, q=FAKE, lens=FAKE, B=64, most=8192, out=FAKE, ws=FAKE, size=need):
        return status(G.g4_attn_decode_mods, p or params(), t or table(8192, 64), 0, mods, q, lens, B, most, out, ws, size,
                      0)

    for kw, want in MODS:
        assert call(mods=G.score_mods(**kw), B=0) == want, kw
    assert call(mods=G.score_mods(key_end=FAKE), B=0) == G.G4_ERR_INVALID_ARG
    assert call(size=need - 1) == G.G4_ERR_WORKSPACE
    for kw in (dict(ws=None), dict(ws=FAKE + 8), dict(q=None), dict(lens=None), dict(out=None), dict(q=FAKE + 8), dict(B=-1)):
        assert call(**kw) == G.G4_ERR_INVALID_ARG, kw
    assert call(B=65) == G.G4_ERR_CAPACITY and call(most=0) == G.G4_ERR_CAPACITY and call(most=8193) == G.G4_ERR_CAPACITY
    assert call(t=table(512, 64, ring=True), most=100000, B=0) == G.G4_OK


def test_mods_and_axes_hold_on_to_what_they_name():
    import gc
    m = G.score_mods(30.0, torch.ones(8), torch.zeros(3, dtype=torch.int32))
    assert m.tensors[0].data_ptr() == m.slopes and m.tensors[1].data_ptr() == m.key_begin and m.key_end is None
    axes = G.rope_axes(2, [1, 0, 1], 8, [0.5, 0.25, 0.125])
    gc.collect()
    assert axes.axis[:4] == [1, 0, 1, 0] and axes.inv_freq[:4] == [0.5, 0.25, 0.125, 0.0]
    for kw in (dict(slopes=torch.ones(8).double()), dict(key_begin=torch.zeros(3)), dict(key_end=torch.zeros(3).long()),
               dict(slopes=torch.ones(16)[::2])):
        with pytest.raises(ValueError):
            G.score_mods(1.0, **kw)
