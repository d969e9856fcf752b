"""Refusals of the paged 4-bit cache's entry points (no GPU needed: they are
decided before anything is launched)."""

import pytest

from gemma_dual_geometry_gb300 import build as g4build
from gemma_dual_geometry_gb300 import g4attn as G

FAKE = 0x7f0000000000  # aligned, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _lib():
    g4build.build()
    G.lib()


def params(**kw):
    d = dict(layer_type=G.G4_SLIDING, head_dim=256, n_heads=8, n_kv_heads=2, window=512, theta=1e4,
             rotary_fraction=1.0, eps=1e-6, attn_scale=1.0, kv_share_src=-1, dtype=G.G4_BF16)
    d.update(kw)
    return G.layer_params(**d)


def pools(**kw):
    d = dict(data=FAKE, layer_type=G.G4_SLIDING, head_dim=256, n_kv_heads=2, n_blocks=10, block_size=64, k_exp=0)
    d.update(kw)
    t = G.kv4_pool_table(1)
    G.set_kv4_pool(t, 0, **d)
    return t


def status(fn, *args):
    try:
        fn(*args, stream=0)
        return G.G4_OK
    except G.G4Error as e:
        assert G.g4_last_error()
        return e.status


def append(p=None, t=None, layer=0, q=FAKE, k=FAKE, v=FAKE, qw=FAKE, kw=FAKE, pos=FAKE, slots=FAKE, B=1, T=0, qo=FAKE):
    return status(G.g4_kv4_append_normrope, p or params(), t or pools(), layer, q, k, v, qw, kw, pos, slots, B, T, qo)


def gather(p=None, t=None, layer=0, table=FAKE, width=4, start=FAKE, lens=FAKE, B=1, rows=0, k=FAKE, v=FAKE):
    return status(G.g4_kv4_gather, p or params(), t or pools(), layer, table, width, start, lens, B, rows, k, v)


def decode(p=None, t=None, layer=0, q=FAKE, table=FAKE, width=4, lens=FAKE, B=0, most=200, out=FAKE, ws=FAKE, nb=1 << 40):
    return status(G.g4_kv4_attn_decode, p or params(), t or pools(), layer, q, table, width, lens, B, most, out, ws, nb)


def prefill(p=None, t=None, layer=0, q=FAKE, table=FAKE, width=4, start=FAKE, lens=FAKE, B=0, T=5, most=200, out=FAKE,
            ws=FAKE, nb=1 << 40):
    return status(G.g4_kv4_attn_prefill, p or params(), t or pools(), layer, q, table, width, start, lens, B, T, most,
                  out, ws, nb)


@pytest.mark.parametrize("call", [append, gather, decode, prefill])
def test_shared_refusals(call):
    assert call() == G.G4_OK                                     # an empty batch (or no tokens)
    assert call(p=params(head_dim=96)) == G.G4_ERR_UNSUPPORTED
    assert call(p=params(n_heads=12)) == G.G4_ERR_UNSUPPORTED     # group 6
    assert call(p=params(window=0)) == G.G4_ERR_INVALID_ARG
    assert call(p=params(dtype=G.G4_F32)) == G.G4_ERR_UNSUPPORTED
    assert call(p=params(layer_type=G.G4_FULL)) == G.G4_ERR_SHARE_MISMATCH
    assert call(p=params(head_dim=128)) == G.G4_ERR_SHARE_MISMATCH
    assert call(p=params(n_kv_heads=4)) == G.G4_ERR_SHARE_MISMATCH
    assert call(t=pools(block_size=48)) == G.G4_ERR_UNSUPPORTED
    assert call(t=pools(block_size=8)) == G.G4_ERR_UNSUPPORTED
    assert call(t=pools(n_blocks=0)) == G.G4_ERR_INVALID_ARG
    assert call(t=pools(n_blocks=1 << 25)) == G.G4_ERR_INVALID_ARG   # 2^31 positions
    assert call(t=pools(n_blocks=(1 << 25) - 1)) == G.G4_OK
    assert call(t=pools(k_exp=33)) == G.G4_ERR_INVALID_ARG
    assert call(t=pools(k_exp=-33)) == G.G4_ERR_INVALID_ARG
    assert call(t=pools(data=None)) == G.G4_ERR_INVALID_ARG
    assert call(t=pools(data=FAKE + 8)) == G.G4_ERR_INVALID_ARG
    assert call(layer=1) == G.G4_ERR_INVALID_ARG
    assert call(layer=-1) == G.G4_ERR_INVALID_ARG
    assert call(B=-1) == G.G4_ERR_INVALID_ARG


def test_append_refusals():
    for name in ("q", "qw", "kw", "k", "v", "pos", "slots", "qo"):
        assert append(**{name: None}) == G.G4_ERR_INVALID_ARG, name
    for name in ("q", "qw", "kw", "k", "v", "qo"):
        assert append(**{name: FAKE + 4}) == G.G4_ERR_INVALID_ARG, name
    assert append(T=-1) == G.G4_ERR_INVALID_ARG
    assert append(B=1 << 20, T=1 << 20) == G.G4_ERR_INVALID_ARG
    shared = params(kv_share_src=0)
    assert append(p=shared) == G.G4_ERR_INVALID_ARG
    assert append(p=shared, k=None, v=None, kw=None, slots=None) == G.G4_OK
    assert append(p=shared, k=None, v=None, kw=None, layer=3) == G.G4_ERR_INVALID_ARG


def test_gather_refusals():
    for name in ("table", "start", "lens", "k", "v"):
        assert gather(**{name: None}) == G.G4_ERR_INVALID_ARG, name
    assert gather(k=FAKE + 2) == G.G4_ERR_INVALID_ARG
    assert gather(width=0) == G.G4_ERR_INVALID_ARG
    assert gather(width=1 << 25) == G.G4_ERR_INVALID_ARG
    assert gather(rows=-1) == G.G4_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [decode, prefill])
def test_attention_refusals(call):
    for name in ("q", "table", "lens", "out"):
        assert call(**{name: None}) == G.G4_ERR_INVALID_ARG, name
    assert call(q=FAKE + 8) == G.G4_ERR_INVALID_ARG
    assert call(out=FAKE + 8) == G.G4_ERR_INVALID_ARG
    assert call(most=0) == G.G4_ERR_CAPACITY
    assert call(most=257) == G.G4_ERR_CAPACITY        # 4 blocks of 64
    assert call(most=256) == G.G4_OK
    assert call(width=-1) == G.G4_ERR_INVALID_ARG
    full = dict(p=params(layer_type=G.G4_FULL, head_dim=512), t=pools(layer_type=G.G4_FULL, head_dim=512, n_blocks=4000),
                B=1, width=2000, most=100000)
    assert call(nb=16, **full) == G.G4_ERR_WORKSPACE
    assert call(ws=None, **full) == G.G4_ERR_INVALID_ARG
    assert call(ws=FAKE + 8, **full) == G.G4_ERR_INVALID_ARG


def test_decode_refuses_what_32_bits_cannot_count():
    huge = dict(p=params(layer_type=G.G4_FULL), t=pools(layer_type=G.G4_FULL, block_size=128), width=1 << 23)
    assert decode(B=1 << 16, most=1 << 30, **huge) == G.G4_ERR_UNSUPPORTED
    assert decode(B=(1 << 31) - 1, most=1 << 20, **huge) == G.G4_ERR_UNSUPPORTED
    assert decode(B=1 << 14, most=1 << 20, nb=16, **huge) == G.G4_ERR_WORKSPACE   # counted


def test_prefill_refusals():
    assert prefill(start=None) == G.G4_ERR_INVALID_ARG
    assert prefill(T=201) == G.G4_ERR_CAPACITY
    assert prefill(T=-1) == G.G4_ERR_INVALID_ARG
    assert prefill(t=pools(block_size=128), width=1 << 23, most=1 << 30, T=1 << 30) == G.G4_ERR_CAPACITY


def test_workspace_sizes():
    p = params()
    assert G.g4_kv4_decode_workspace_size(p, 64, 100000) == G.g4_kv4_decode_workspace_size(p, 64, 8192)  # the window
    assert G.g4_kv4_decode_workspace_size(params(dtype=G.G4_F32), 64, 100) == 0
    assert G.g4_kv4_decode_workspace_size(p, 0, 100) == 0
    # T + window - 1 rows of K and V per sequence and head, and the sequences' first rows
    assert G.g4_kv4_prefill_workspace_size(p, 3, 100, 5000) == 256 + 2 * 3 * 2 * 611 * 256 * 2
    # but no more than max_seq_len and T positions of padding behind it
    assert G.g4_kv4_prefill_workspace_size(p, 3, 100, 300) == 256 + 2 * 3 * 2 * 400 * 256 * 2
    assert G.g4_kv4_prefill_workspace_size(p, 3, 100, 99) == 0
    assert G.kv4_pool_bytes(10, 2, 64, 256) == 10 * 64 * 2 * 2 * (256 // 2 + 256 // 16)


def assign(B=1, T=1, bs=16, n=10, width=4, **kw):
    names = ("old", "new", "free", "count", "table", "lens", "left", "pos", "slots")
    return status(G.g4_kv4_assign_blocks, B, T, bs, n, width, *(kw.get(x, FAKE) for x in names))


def test_assign_refusals():
    for name in ("old", "new", "free", "count", "table", "lens", "left", "pos", "slots"):
        assert assign(**{name: None}) == G.G4_ERR_INVALID_ARG, name
    assert assign(bs=20) == G.G4_ERR_UNSUPPORTED
    assert assign(n=0) == G.G4_ERR_INVALID_ARG
    assert assign(n=1 << 28) == G.G4_ERR_INVALID_ARG
    assert assign(width=0) == G.G4_ERR_INVALID_ARG
    assert assign(B=-1) == G.G4_ERR_INVALID_ARG
    assert assign(T=-1) == G.G4_ERR_INVALID_ARG
    assert assign(B=8193) == G.G4_ERR_UNSUPPORTED
    assert assign(B=8192, width=1 << 18) == G.G4_ERR_INVALID_ARG
    assert assign(B=8192, T=1 << 18) == G.G4_ERR_INVALID_ARG
