"""Parity of the paged 4-bit KV cache (g4_kv4_*) against the float64 oracles.

Exact: the pool's bytes after an append, what gather reads back, block tables
and slots.  Attention: |error| <= 2^-8 |out| + c sum_j p_j |v_j|.  The first
term is the output's rounding to bf16 (half a step, eps / 2).  c covers the
relative errors of the weights p_j.  Decode: a probability is rounded to fp16
and so is its product with a scale (2^-11 each, and the subnormal range starts
2^-18 below the reference, where a rounding of 2^-24 - 2^-25 of 2^-14 is
relative to weights of that size); scores of |s| <= 60 (log2) from float32 sums
of hd exact products with partial sums below 16 |s|: hd 2^-24 16 60 / 16
<= 2^-9.1 at hd 512 were every rounding one way; a bound of 2^-9 on the sum of
both needs the roundings of the score to be half that, so c = 2^-8 is used.
(fp16's subnormal range adds an absolute term: kv4_common.assert_within.)
Prefill rounds its probabilities to bf16 (2^-8) and sums the rounded or the
unrounded ones (2^-8 again): c = 2^-7.
"""

import numpy as np
import pytest

from gemma_dual_geometry_gb300 import build as g4build

from kv4_common import (DEV, G, K, O, Pool, W, assert_within, attention_and_scale, bf16_normal, f64, geometry, i32,
                        params_of, torch)

pytestmark = pytest.mark.gpu

C_DECODE, C_PREFILL = 2.0 ** -8, 2.0 ** -7
# (layer type, head_dim, H, Hkv, window)
GEOS = [(W.SLIDING, 256, 8, 2, 40), (W.FULL, 512, 8, 2, 0), (W.FULL, 128, 8, 1, 0), (W.SLIDING, 64, 3, 3, 17),
        (W.FULL, 256, 4, 2, 0), (W.SLIDING, 512, 4, 4, 33)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    g4build.build()
    G.lib()
    yield
    assert G.g4_take_device_error() == 0


def geo_of(g):
    return geometry(g[0], g[1], H=g[2], Hkv=g[3], window=g[4])


# ---------------------------------------------------------------- block assignment

def assign_gpu(old, new, T, bs, n, free, count, table, alias=False):
    B, width = table.shape
    d_old, d_new, d_free, d_count, d_table = i32(old), i32(new), i32(free), i32([count]), i32(table)
    lens = d_old if alias else i32(np.zeros(B))
    left = d_count if alias else i32([0])
    pos, slots = i32(np.zeros((B, T))), i32(np.zeros((B, T)))
    calls = 1 if alias else 2  # a repeated call repeats its results
    for _ in range(calls):
        G.g4_kv4_assign_blocks(B, T, bs, n, width, d_old, d_new, d_free, d_count, d_table, lens, left, pos, slots)
    return [x.cpu().numpy() for x in (d_table, d_free, left, lens, pos, slots)]


@pytest.mark.parametrize("B,T,bs,width,short", [(1, 1, 16, 1, False), (5, 7, 16, 9, True), (64, 1, 64, 12, False),
                                                (513, 3, 32, 6, True), (700, 70, 16, 9, True), (8192, 1, 16, 3, False),
                                                (3, 9000, 128, 90, False), (40, 2048, 64, 70, True), (9, 0, 16, 4, True)])
@pytest.mark.parametrize("alias", [False, True])
def test_assign_blocks(B, T, bs, width, short, alias):
    rng = np.random.default_rng(B * 31 + T)
    cap = width * bs
    n = B * width + 5
    lens = rng.integers(0, cap + 1, B)
    table = np.full((B, width), -1)
    order = rng.permutation(n)
    at = 0
    for b in range(B):
        k = -(-int(lens[b]) // bs)
        table[b, :k] = order[at:at + k]
        at += k
    free = np.full(n, -1)
    count = n - at if not short else min(n - at, 2)
    free[:count] = order[at:at + count]
    kind = rng.random(B)
    new = np.where(kind < 0.2, 0, np.where(kind < 0.3, lens // 2, lens + rng.integers(0, T + 3, B)))
    new[:1] = cap + 100  # clamped
    want = K.assign_blocks(lens, new, T, bs, n, free, count, table)
    got = assign_gpu(lens, new, T, bs, n, free, count, table, alias)
    for name, g, w in zip(("table", "free", "count", "lens", "positions", "slots"), got, want):
        assert np.array_equal(g.ravel(), np.asarray(w).ravel()), name


def test_assign_no_sequences():
    free, count, out = i32([3, 1, 2, 0]), i32([3]), i32([9])
    e = i32(np.zeros(1))
    G.g4_kv4_assign_blocks(0, 1, 16, 4, 1, e, e, free, count, e, e, out, e, e)
    assert out.item() == 3 and free.tolist() == [3, 1, 2, 0]


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("geo", GEOS)
@pytest.mark.parametrize("B,T,bs,k_exp", [(3, 1, 16, 0), (2, 37, 32, -2), (1, 150, 128, 3), (7, 18, 64, 0)])
def test_append_bytes(geo, B, T, bs, k_exp):
    g = geo_of(geo)
    hd, H, Hkv = g["head_dim"], g["n_heads"], g["n_kv_heads"]
    rng = np.random.default_rng(hd + T)
    start = rng.integers(0, 100, B)
    start[1:3] = start[0]        # neighbours that share a cos/sin table
    pool = Pool(g, B, 100 + T, bs, seed=hd + B, k_exp=k_exp)
    x = {c: bf16_normal((B, T, h, hd), 50 + i) for i, (c, h) in enumerate((("q", H), ("k", Hkv), ("v", Hkv)))}
    x["k"][0, 0, 0, 3] = 1e-30   # a tiny value, and an all-zero row
    x["v"][0, 0, 0] = 0
    qw, kw = W.norm_weight(hd, 7), W.norm_weight(hd, 8)
    kw[16:32] = 0.0              # a block of zeros: scale 0
    pos = start[:, None] + np.arange(T)[None, :]
    slots = np.array([[pool.slot(b, p) for p in pos[b]] for b in range(B)])
    if T > 1:
        slots[0, 1] = -1
        slots[B - 1, T - 1] = pool.n * bs  # outside the pool
    pool.to_device()
    q = x["q"].to(DEV)
    q_out = torch.empty_like(q)
    G.g4_kv4_append_normrope(params_of(g), pool.pools, 0, q, x["k"].to(DEV), x["v"].to(DEV), qw.to(DEV), kw.to(DEV),
                             i32(pos), i32(slots), B, T, q_out)
    want = pool.data.copy()
    kn, vn = O.normrope_kv(f64(x["k"]), f64(x["v"]), f64(kw), pos, hd, g["theta"], g["rotary_fraction"], g["eps"])
    kn, vn = O.round_bf16(kn), O.round_bf16(vn)
    for b in range(B):
        for t in range(T):
            if 0 <= slots[b, t] < pool.n * bs:
                for h in range(Hkv):
                    K.write_slot(want, int(slots[b, t]), h, kn[b, t, h], vn[b, t, h], bs, k_exp)
    got = pool.d.cpu().numpy()
    assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ"
    ref_q = O.round_bf16(O.normrope_q(f64(x["q"]), f64(qw), pos, hd, g["theta"], g["rotary_fraction"], g["eps"]))
    assert np.array_equal(f64(q_out), ref_q)


def test_append_non_finite_rows_stand_for_nans():
    g = geo_of(GEOS[0])
    pool = Pool(g, 1, 16, 16, seed=1).to_device()
    k, v = (bf16_normal((1, 2, 2, 256), s) for s in (1, 2))
    k[0, 0, 1, 9] = float("nan")
    v[0, 1, 0, 0] = float("inf")
    q = bf16_normal((1, 2, 8, 256), 3).to(DEV)
    w = W.norm_weight(256, 4).to(DEV)
    slots = [[pool.slot(0, 0), pool.slot(0, 1)]]
    G.g4_kv4_append_normrope(params_of(g), pool.pools, 0, q, k.to(DEV), v.to(DEV), w, w, i32([[0, 1]]), i32(slots), 1, 2,
                             torch.empty_like(q))
    ko, vo = (torch.empty((1, 2, 2, 256), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    G.g4_kv4_gather(params_of(g), pool.pools, 0, pool.d_table, pool.per, i32([0]), i32([2]), 1, 2, ko, vo)
    kb, vb = torch.isnan(ko)[0], torch.isnan(vo)[0]   # [head][position][element]
    assert kb[1, 0].any() and not kb[0].any() and not kb[1, 1].any()
    assert vb[0, 1].any() and not vb[1].any() and not vb[0, 0].any()


def test_append_shared_layer_ropes_q_only():
    g = geo_of(GEOS[0])
    pool = Pool(g, 1, 32, 16, seed=2).to_device()
    q = bf16_normal((1, 5, 8, 256), 3)
    w = W.norm_weight(256, 4)
    out = torch.empty_like(q, device=DEV)
    pools = G.kv4_pool_table(2)
    pools[0] = pool.pools[0]
    G.g4_kv4_append_normrope(params_of(g, src=0), pools, 1, q.to(DEV), None, None, w.to(DEV), None,
                             i32([[0, 1, 2, 70000, -1]]), None, 1, 5, out)
    ref = O.round_bf16(O.normrope_q(f64(q), f64(w), np.array([[0, 1, 2, 70000, -1]]), 256, 1e4, 1.0, g["eps"]))
    assert np.array_equal(f64(out), ref)
    assert np.array_equal(pool.d.cpu().numpy(), pool.data)


# ---------------------------------------------------------------- gather

@pytest.mark.parametrize("geo", GEOS)
@pytest.mark.parametrize("bs,k_exp", [(16, 0), (64, -3), (128, 2)])
def test_gather_exact(geo, bs, k_exp):
    g = geo_of(geo)
    hd, Hkv = g["head_dim"], g["n_kv_heads"]
    B, rows = 5, 77
    lens = np.array([0, 1, 100, 150, 33])
    start = np.array([0, 0, 37, 90, -20])
    pool = Pool(g, B, 150, bs, seed=hd, k_exp=k_exp).fill(lens, 5)
    if pool.per > 1:
        pool.table[3, 1] = pool.n + 4   # an id outside the pool: zeros
    pool.to_device()
    k, v = (torch.full((B, Hkv, rows, hd), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    G.g4_kv4_gather(params_of(g), pool.pools, 0, pool.d_table, pool.per, i32(start), i32(lens), B, rows, k, v)
    for b in range(B):
        at = start[b] + np.arange(rows)
        for h in range(Hkv):
            rk, rv = K.read_rows(pool.data, pool.table[b], h, at, bs, k_exp)
            held = ((at >= 0) & (at < lens[b]))[:, None]
            for got, ref in ((k, rk), (v, rv)):
                ref = np.where(held & ~np.isnan(ref), ref, 0.0)
                assert np.array_equal(f64(got[b, h]), ref), (b, h)


# ---------------------------------------------------------------- decode

def decode_gpu(g, pool, q, lens, most=None, out=None, ws=None):
    p = params_of(g)
    most = most or pool.per * pool.bs
    nb = G.g4_kv4_decode_workspace_size(p, pool.B, most)
    ws = torch.zeros(max(16, nb), dtype=torch.uint8, device=DEV) if ws is None else ws
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV) if out is None else out
    G.g4_kv4_attn_decode(p, pool.pools, 0, q.to(DEV), pool.d_table, pool.per, i32(lens), pool.B, most, out, ws, nb)
    return out


@pytest.mark.parametrize("geo", GEOS + [(W.FULL, 64, 8, 1, 0), (W.FULL, 128, 2, 2, 0), (W.SLIDING, 128, 4, 1, 1),
                                        (W.SLIDING, 256, 8, 1, 16)])
@pytest.mark.parametrize("bs,k_exp", [(16, 0), (32, 2), (128, -3)])
def test_decode(geo, bs, k_exp):
    g = geo_of(geo)
    hd, H, Hkv = g["head_dim"], g["n_heads"], g["n_kv_heads"]
    lens = np.array([0, 1, 15, 16, 17, 31, 64, 65, 200, 333])
    pool = Pool(g, len(lens), 333, bs, seed=hd + H, k_exp=k_exp).fill(lens, 9).to_device()
    q = (bf16_normal((len(lens), H, hd), 11).float() * 2.0 ** -k_exp).to(torch.bfloat16)
    out = f64(decode_gpu(g, pool, q, lens))
    k, v = pool.rows(lens, 333)
    ref, mag = attention_and_scale(f64(q)[:, None], k, v, (lens - 1)[:, None], lens, Hkv, g)
    assert (out[0] == 0).all()
    assert_within(out, ref[:, 0], mag[:, 0], C_DECODE, f"{geo} bs {bs}", keys=333)


@pytest.mark.parametrize("B,L,hd", [(1, 4000, 512), (2, 5001, 256), (3, 3111, 128), (1, 2500, 64)])
def test_decode_many_splits(B, L, hd):
    g = geometry(W.FULL, hd, H=4, Hkv=1)
    lens = np.array([L - 700 * i for i in range(B)])
    pool = Pool(g, B, L, 64, seed=hd).fill(lens, 3).to_device()
    q = bf16_normal((B, 4, hd), 12)
    p = params_of(g)
    assert G.g4_kv4_decode_workspace_size(p, B, pool.per * 64) > 0
    nb = G.g4_kv4_decode_workspace_size(p, B, pool.per * 64)
    ws = torch.zeros(nb, dtype=torch.uint8, device=DEV)
    a = decode_gpu(g, pool, q, lens, ws=ws)
    first = f64(a)
    k, v = pool.rows(lens, L)
    ref, mag = attention_and_scale(f64(q)[:, None], k, v, (lens - 1)[:, None], lens, 1, g)
    assert_within(first, ref[:, 0], mag[:, 0], C_DECODE, keys=L)
    # the workspace is ready for the next call, whose lengths differ; and the bits repeat
    short = np.maximum(1, lens - 1900)
    k, v = pool.rows(short, L)
    ref, mag = attention_and_scale(f64(q)[:, None], k, v, (short - 1)[:, None], short, 1, g)
    assert_within(f64(decode_gpu(g, pool, q, short, ws=ws)), ref[:, 0], mag[:, 0], C_DECODE, keys=L)
    assert np.array_equal(f64(decode_gpu(g, pool, q, lens, ws=ws)), first)


def test_decode_extreme_queries():
    """q far from unit size (its fp16 form is scaled by a power of two per head), and peaked rows."""
    g = geometry(W.FULL, 128, H=8, Hkv=1)
    lens = np.array([130])
    pool = Pool(g, 1, 130, 16, seed=5).fill(lens, 6).to_device()
    q = bf16_normal((1, 8, 128), 13).float()
    for h, f in enumerate((1e-30, 1e-6, 1e-3, 1.0, 4.0, 0.0, 2.0 ** -14, 3.0)):
        q[0, h] *= f
    q = q.to(torch.bfloat16)
    out = f64(decode_gpu(g, pool, q, lens))
    k, v = pool.rows(lens, 130)
    ref, mag = attention_and_scale(f64(q)[:, None], k, v, (lens - 1)[:, None], lens, 1, g)
    assert_within(out, ref[:, 0], mag[:, 0], C_DECODE, keys=130)
    # scores far below zero (log2 around -1e32) still weigh against each other: one key is all of it
    one = Pool(g, 1, 16, 16, seed=5).fill([1], 6).to_device()
    big = torch.full((1, 8, 128), -(2.0 ** 100), dtype=torch.bfloat16)
    k, v = one.rows([1], 16)
    big = torch.sign(torch.from_numpy(k[0, :, 0])).to(torch.bfloat16) * big
    assert_within(f64(decode_gpu(g, one, big, [1])), np.repeat(v[:, :, 0], 8, 1), np.abs(np.repeat(v[:, :, 0], 8, 1)), C_DECODE)


def test_decode_absent_blocks_and_clamped_lengths():
    """Ids outside the pool hold no keys; entries outside the window are not read; lengths are clamped."""
    g = geometry(W.FULL, 256, H=4, Hkv=2)
    lens = np.array([96, 96, 96])
    pool = Pool(g, 3, 96, 32, seed=8).fill(lens, 2)
    k, v = pool.rows(lens, 96)
    pool.table[0, 1], pool.table[1, :] = -1, pool.n
    pool.to_device()
    q = bf16_normal((3, 4, 256), 14)
    out = f64(decode_gpu(g, pool, q, [96, 96, 10 ** 9]))
    keep = np.r_[0:32, 64:96]
    ref, mag = attention_and_scale(f64(q)[:1, None], k[:1, :, keep], v[:1, :, keep], np.array([[63]]), [64], 2, g)
    assert_within(out[:1], ref[:, 0], mag[:, 0], C_DECODE, keys=64)
    assert (out[1] == 0).all()
    ref, mag = attention_and_scale(f64(q)[2:, None], k[2:], v[2:], np.array([[95]]), [96], 2, g)
    assert_within(out[2:], ref[:, 0], mag[:, 0], C_DECODE, keys=96)
    assert (f64(decode_gpu(g, pool, q, [-5, 0, -2 ** 31])) == 0).all()
    # a sliding layer whose blocks before the window have been given away
    g = geometry(W.SLIDING, 256, H=4, Hkv=2, window=20)
    pool = Pool(g, 1, 96, 16, seed=8).fill([96], 2)
    k, v = pool.rows([96], 96)
    pool.table[0, :4] = -1
    pool.to_device()
    out = f64(decode_gpu(g, pool, q[:1], [96]))
    ref, mag = attention_and_scale(f64(q)[:1, None], k, v, np.array([[95]]), [96], 2, g)
    assert_within(out, ref[:, 0], mag[:, 0], C_DECODE, keys=20)


# ---------------------------------------------------------------- prefill

@pytest.mark.parametrize("geo", GEOS)
@pytest.mark.parametrize("T,bs,k_exp", [(1, 16, 0), (40, 32, -2), (200, 128, 1)])
def test_prefill(geo, T, bs, k_exp):
    g = geo_of(geo)
    hd, H, Hkv = g["head_dim"], g["n_heads"], g["n_kv_heads"]
    start = np.array([0, 1, 70, 133])
    B, cap = 4, 133 + T
    lens = start + T
    lens[2] -= T // 3   # padding behind the sequence
    pool = Pool(g, B, cap, bs, seed=hd + T, k_exp=k_exp).fill(lens, 4).to_device()
    q = (bf16_normal((B, T, H, hd), 15).float() * 2.0 ** -k_exp).to(torch.bfloat16)
    p = params_of(g)
    nb = G.g4_kv4_prefill_workspace_size(p, B, T, cap)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device=DEV)   # NaNs
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
    G.g4_kv4_attn_prefill(p, pool.pools, 0, q.to(DEV), pool.d_table, pool.per, i32(start), i32(lens), B, T, cap, out, ws,
                          nb)
    k, v = pool.rows(lens, cap)
    pos = start[:, None] + np.arange(T)[None, :]
    ref, mag = attention_and_scale(f64(q), k, v, pos, start + T, Hkv, g)
    assert_within(f64(out), ref, mag, C_PREFILL, f"{geo} T {T}")


@pytest.mark.parametrize("geo", GEOS)
def test_prefill_padding_past_the_table(geo):
    """A padded batch whose sequences end at, near and before the table's end: the new tokens keep their
    positions, whatever of the padding would lie past the end."""
    g = geo_of(geo)
    hd, H, Hkv = g["head_dim"], g["n_heads"], g["n_kv_heads"]
    T, cap = 150, 160
    start = np.array([158, 160, 20, 0, 100])
    fresh = np.array([2, 0, 140, 150, 1])
    B, lens = 5, start + fresh
    pool = Pool(g, B, cap, 32, seed=hd).fill(lens, 4).to_device()
    q = bf16_normal((B, T, H, hd), 15)
    p = params_of(g)
    nb = G.g4_kv4_prefill_workspace_size(p, B, T, cap)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device=DEV)   # NaNs
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
    G.g4_kv4_attn_prefill(p, pool.pools, 0, q.to(DEV), pool.d_table, pool.per, i32(start), i32(lens), B, T, cap, out, ws,
                          nb)
    assert bool(torch.isfinite(out).all())
    k, v = pool.rows(lens, cap)
    for b in range(B):
        n = fresh[b]
        if n == 0:
            continue
        one = slice(b, b + 1)
        pos = (start[b] + np.arange(n))[None]
        ref, mag = attention_and_scale(f64(q)[one, :n], k[one], v[one], pos, lens[one], Hkv, g)
        assert_within(f64(out)[one, :n], ref, mag, C_PREFILL, f"{geo} sequence {b}")


@pytest.mark.parametrize("hd,H,window", [(512, 4, 0), (64, 2, 0), (256, 8, 9000)])
def test_prefill_under_a_wide_bound(hd, H, window):
    """The same result whatever the bound on the lengths, far above them too (and the gather's CTAs take turns)."""
    g = geometry(W.SLIDING if window else W.FULL, hd, H=H, Hkv=2, window=window)
    T, B, bs = 33, 4, 128
    start = np.array([300, 0, 77, 512])
    lens = start + T
    pool = Pool(g, B, 640, bs, seed=hd).fill(lens, 4).to_device()
    p, q = params_of(g), bf16_normal((B, T, H, hd), 15).to(DEV)
    outs = []
    for width in (pool.per, 300):
        table = torch.full((B, width), 1 << 30, dtype=torch.int32, device=DEV)
        table[:, :pool.per] = pool.d_table
        most = width * bs
        nb = G.g4_kv4_prefill_workspace_size(p, B, T, most)
        ws = torch.full((nb,), 255, dtype=torch.uint8, device=DEV)
        outs.append(torch.empty_like(q))
        G.g4_kv4_attn_prefill(p, pool.pools, 0, q, table, width, i32(start), i32(lens), B, T, most, outs[-1], ws, nb)
    assert torch.equal(*outs)
    k, v = pool.rows(lens, 640)
    ref, mag = attention_and_scale(f64(q), k, v, start[:, None] + np.arange(T), lens, 2, g)
    assert_within(f64(outs[1]), ref, mag, C_PREFILL)


def test_gather_of_many_rows():
    """More rows than a launch has CTAs for, from before a sequence's first position to behind its last."""
    g = geometry(W.FULL, 512, H=2, Hkv=2)
    lens, start, rows = np.array([14000, 13990, 3000]), np.array([-5, 100, 7]), 14001
    pool = Pool(g, 3, 14000, 64, seed=5).to_device()   # random bytes
    k, v = (torch.empty((3, 2, rows, 512), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    G.g4_kv4_gather(params_of(g), pool.pools, 0, pool.d_table, pool.per, i32(start), i32(lens), 3, rows, k, v)
    for b in range(3):
        outside = np.ones(rows, bool)
        outside[max(0, -start[b]):lens[b] - start[b]] = False
        for x in (k, v):
            assert not x[b][:, torch.from_numpy(outside).to(DEV)].any()
        some = np.unique(np.concatenate([np.arange(0, lens[b], 211), np.arange(max(0, start[b]), max(0, start[b]) + 20),
                                         np.arange(lens[b] - 20, lens[b])]))
        some = some[(some >= start[b]) & (some < start[b] + rows)]
        for h in range(2):
            for got, want in zip((k, v), K.read_rows(pool.data, pool.table[b], h, some, 64)):
                assert np.array_equal(f64(got[b, h, torch.from_numpy(some - start[b]).to(DEV)]), want, equal_nan=True)


# ---------------------------------------------------------------- as they are used

def test_lifecycle_under_graphs():
    """Prompts, decode steps and ends of sequences through all five operators on two streams' worth of calls:
    assignment, append and decode captured once and replayed with changing lengths, two graphs with a
    workspace each, against a float64 model that keeps rows in lists."""
    g = geometry(W.SLIDING, 128, H=4, Hkv=2, window=30)
    p = params_of(g)
    B, bs, width, n, hd = 4, 16, 8, 14, 128
    data = torch.randint(0, 256, (n, 2, 1, 18 * hd), dtype=torch.uint8, device=DEV)
    pools = G.kv4_pool_table(1)
    G.set_kv4_pool(pools, 0, data, W.SLIDING, hd, 2, n, bs)
    table, free, count = i32(np.full((B, width), -1)), i32(np.arange(n)), i32([n])
    lens, want = i32(np.zeros(B)), i32(np.zeros(B))
    qw, kw = W.norm_weight(hd, 1).to(DEV), W.norm_weight(hd, 2).to(DEV)
    stream = torch.cuda.Stream()
    rows = [[] for _ in range(B)]  # (k, v) rows as stored
    model = dict(table=np.full((B, width), -1), free=np.arange(n), count=n, lens=np.zeros(B, int))

    def make(T):
        z = dict(T=T, q=torch.zeros((B, T, 4, hd), dtype=torch.bfloat16, device=DEV))
        z["k"], z["v"] = (torch.zeros((B, T, 2, hd), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        z["pos"], z["slots"] = i32(np.zeros((B, T))), i32(np.zeros((B, T)))
        z["start"] = i32(np.zeros(B))
        z["qo"], z["out"] = torch.empty_like(z["q"]), torch.empty_like(z["q"])
        cap = width * bs
        z["nb"] = (G.g4_kv4_decode_workspace_size(p, B, cap) if T == 1 else
                   G.g4_kv4_prefill_workspace_size(p, B, T, cap))
        z["ws"] = torch.zeros(max(16, z["nb"]), dtype=torch.uint8, device=DEV)
        return z

    def calls(z):
        T = z["T"]
        z["start"].copy_(lens)
        G.g4_kv4_assign_blocks(B, T, bs, n, width, lens, want, free, count, table, lens, count, z["pos"], z["slots"])
        G.g4_kv4_append_normrope(p, pools, 0, z["q"], z["k"], z["v"], qw, kw, z["pos"], z["slots"], B, T, z["qo"])
        if T == 1:
            G.g4_kv4_attn_decode(p, pools, 0, z["qo"], table, width, lens, B, width * bs, z["out"], z["ws"], z["nb"])
        else:
            G.g4_kv4_attn_prefill(p, pools, 0, z["qo"], table, width, z["start"], lens, B, T, width * bs, z["out"],
                                  z["ws"], z["nb"])

    steps = {T: make(T) for T in (1, 24)}
    with torch.cuda.stream(stream):
        for z in steps.values():   # once outside the capture (with nothing wanted), as a program warms up
            calls(z)
        stream.synchronize()
        for z in steps.values():
            z["graph"] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(z["graph"], stream=stream):
                calls(z)
        rng = np.random.default_rng(0)
        for step in range(14):
            T = 24 if step in (0, 5, 6) else 1
            z = steps[T]
            target = np.minimum(model["lens"] + (rng.integers(1, T + 1, B) if T > 1 else 1), width * bs)
            if step in (4, 9):
                target[step % B] = 0
            for name, h in (("q", 4), ("k", 2), ("v", 2)):
                z[name].copy_(bf16_normal((B, T, h, hd), 100 * step + h + ord(name)))
            want.copy_(i32(target))
            z["graph"].replay()
            old = model["lens"]
            table_, free_, count_, lens_, pos, slots = K.assign_blocks(old, target, T, bs, n, model["free"],
                                                                       model["count"], model["table"])
            model = dict(table=table_, free=free_, count=count_, lens=lens_)
            stream.synchronize()
            for name, got, ref in (("table", table, table_), ("free", free, free_), ("count", count, count_),
                                   ("lens", lens, lens_), ("pos", z["pos"], pos), ("slots", z["slots"], slots)):
                assert np.array_equal(got.cpu().numpy().ravel(), np.asarray(ref).ravel()), (step, name)
            kn, vn = O.normrope_kv(f64(z["k"]), f64(z["v"]), f64(kw), pos, hd, g["theta"], 1.0, g["eps"])
            kn, vn = (K.values(*K.quantise(O.round_bf16(x))) for x in (kn, vn))
            qn = O.round_bf16(O.normrope_q(f64(z["q"]), f64(qw), pos, hd, g["theta"], 1.0, g["eps"]))
            for b in range(B):
                del rows[b][lens_[b]:]
                for t in range(max(0, lens_[b] - old[b])):
                    rows[b].append((kn[b, t], vn[b, t]))
                m = len(rows[b])
                assert m == lens_[b]
                fresh = lens_[b] - old[b] if T > 1 else 1
                if m == 0 or fresh <= 0:
                    if m == 0 and T == 1:
                        assert (f64(z["out"][b]) == 0).all()
                    continue
                k = np.stack([r[0] for r in rows[b]], 1)[None]
                v = np.stack([r[1] for r in rows[b]], 1)[None]
                if T == 1:
                    q, at = qn[b:b + 1], np.array([[m - 1]])
                else:
                    q, at = qn[b:b + 1, :fresh], (old[b] + np.arange(fresh))[None]
                ref, mag = attention_and_scale(q, k, v, at, np.array([m]), 2, g)
                assert_within(f64(z["out"][b:b + 1, :fresh]), ref, mag, C_DECODE if T == 1 else C_PREFILL, f"step {step}", keys=m if T == 1 else 0)


@pytest.mark.parametrize("geo", [(W.FULL, 256, 8, 2, 0), (W.FULL, 128, 8, 1, 0), (W.FULL, 512, 2, 2, 0)])
def test_decode_nan_stays_in_its_head_and_large_scales(geo):
    """A NaN in q or in a visible row reaches its own heads only; value scales up to e4m3's largest do not
    overflow the fp16 products (rows of the append never come near: their mean square is 1)."""
    g = geo_of(geo)
    hd, H, Hkv = g["head_dim"], g["n_heads"], g["n_kv_heads"]
    lens = np.array([90, 90])
    pool = Pool(g, 2, 90, 32, seed=3).fill(lens, 4)
    kc, ks, vc, vs = K.record_offsets(hd)
    for b in range(2):
        for p in range(90):
            rec = pool.data[pool.table[b, p // 32], :, p % 32 // 16]
            rec[:, vs[p % 16, 0::16]] = 126 - p % 3   # 448, 416, 384
    q = bf16_normal((2, H, hd), 5)
    q[1, H - 1, 7] = float("nan")
    if Hkv > 1:
        pool.data[pool.table[0, 1], 0, 0, ks[5, 32]] = 127   # position 37 of sequence 0, kv head 0
    pool.to_device()
    out = f64(decode_gpu(g, pool, q, lens))
    bad = np.zeros((2, H), bool)
    bad[1, H - 1] = True
    if Hkv > 1:
        bad[0, :H // Hkv] = True
    assert np.isnan(out[bad]).all()
    k, v = pool.rows(lens, 90)
    ok = ~bad
    with np.errstate(invalid="ignore"):
        ref, mag = attention_and_scale(f64(q)[:, None], k, v, (lens - 1)[:, None], lens, Hkv, g)
    # (keys * 2^-25 of kv4_common.assert_within is for scales up to 1.6)
    assert_within(out[ok], ref[:, 0][ok], mag[:, 0][ok], C_DECODE, keys=90 * 449 / 2.6)


def test_decode_one_sequence_over_the_whole_gpu():
    """One kv head of one long sequence: every CTA holds a part, three levels of merges."""
    g = geometry(W.FULL, 64, H=2, Hkv=1)
    L = 60000
    pool = Pool(g, 1, L, 128, seed=4).fill([L], 5).to_device()
    q = bf16_normal((1, 2, 64), 6)
    k, v = pool.rows([L], L)
    ref, mag = attention_and_scale(f64(q)[:, None], k, v, np.array([[L - 1]]), [L], 1, g)
    nb = G.g4_kv4_decode_workspace_size(params_of(g), 1, pool.per * 128)
    ws = torch.zeros(nb, dtype=torch.uint8, device=DEV)
    first = f64(decode_gpu(g, pool, q, [L], ws=ws))
    assert_within(first, ref[:, 0], mag[:, 0], C_DECODE, keys=L)
    assert np.array_equal(f64(decode_gpu(g, pool, q, [L], ws=ws)), first)


def test_offsets_past_32_bits():
    """A pool of 5.3 GB: rows in its last blocks are those of a small pool, byte for byte, and attend alike."""
    g = geometry(W.FULL, 512, H=8, Hkv=2)
    p = params_of(g)
    n, bs, T = 36000, 128, 200
    q, k, v = (bf16_normal((1, T, h, 512), s).to(DEV) for h, s in ((8, 1), (2, 2), (2, 3)))
    qw, kw = W.norm_weight(512, 4).to(DEV), W.norm_weight(512, 5).to(DEV)
    pos = np.arange(T)[None]
    res = []
    for blocks, count in (([[1, 0]], 2), ([[n - 1, n - 2]], n)):
        data = torch.zeros(G.kv4_pool_bytes(count, 2, bs, 512), dtype=torch.uint8, device=DEV)
        pools = G.kv4_pool_table(1)
        G.set_kv4_pool(pools, 0, data, W.FULL, 512, 2, count, bs)
        slots = np.asarray(blocks)[0][pos // bs] * bs + pos % bs
        qo, out = torch.empty_like(q), torch.empty_like(q)
        G.g4_kv4_append_normrope(p, pools, 0, q, k, v, qw, kw, i32(pos), i32(slots), 1, T, qo)
        table = i32(blocks)
        nb = G.g4_kv4_decode_workspace_size(p, 1, T)
        ws = torch.zeros(nb, dtype=torch.uint8, device=DEV)
        dec = torch.empty((1, 8, 512), dtype=torch.bfloat16, device=DEV)
        G.g4_kv4_attn_decode(p, pools, 0, qo[:, -1].contiguous(), table, 2, i32([T]), 1, T, dec, ws, nb)
        nb = G.g4_kv4_prefill_workspace_size(p, 1, T, T)
        ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
        G.g4_kv4_attn_prefill(p, pools, 0, qo, table, 2, i32([0]), i32([T]), 1, T, T, out, ws, nb)
        ko, vo = (torch.empty((1, 2, T, 512), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        G.g4_kv4_gather(p, pools, 0, table, 2, i32([0]), i32([T]), 1, T, ko, vo)
        res.append((dec, out, ko, vo))
        del data
    for a, b in zip(*res):
        assert torch.equal(a, b) and torch.isfinite(a).all()
    torch.cuda.empty_cache()


def test_decode_right_behind_the_kernel_that_sets_the_lengths():
    """Lengths change in the kernel launched just before, with nothing waited for in between."""
    g = geometry(W.FULL, 128, H=4, Hkv=2)
    p = params_of(g)
    B, bs, steps = 3, 128, 20
    pool = Pool(g, B, bs, bs, seed=2).fill([bs] * B, 3).to_device()
    q = bf16_normal((B, 4, 128), 4).to(DEV)
    nb = G.g4_kv4_decode_workspace_size(p, B, bs)
    ws = torch.zeros(nb, dtype=torch.uint8, device=DEV)
    lens, left, free = i32([3, 40, 100]), i32([0]), i32(np.zeros(pool.n))
    want = [i32([3 + i, 40 + i, 100 + i]) for i in range(1, steps + 1)]
    pos, slots = i32(np.zeros((B, 1))), i32(np.zeros((B, 1)))
    outs = [torch.empty_like(q) for _ in want]
    for w, out in zip(want, outs):   # (no sequence leaves its first block)
        G.g4_kv4_assign_blocks(B, 1, bs, pool.n, 1, lens, w, free, left, pool.d_table, lens, left, pos, slots)
        G.g4_kv4_attn_decode(p, pool.pools, 0, q, pool.d_table, 1, lens, B, bs, out, ws, nb)
    for w, out in zip(want, outs):
        torch.cuda.synchronize()
        again = torch.empty_like(q)
        G.g4_kv4_attn_decode(p, pool.pools, 0, q, pool.d_table, 1, w, B, bs, again, ws, nb)
        assert torch.equal(out, again)


@pytest.mark.parametrize("hd,B", [(512, 200), (256, 290), (256, 150), (64, 200)])
def test_decode_one_long_among_many_short(hd, B):
    """Shares that are not cut at units, with a unit spread over many of them (512, 290 of 256); the others are cut."""
    g = geometry(W.FULL, hd, H=2, Hkv=2)
    lens = np.random.default_rng(B).integers(60, 112, B)
    lens[B // 3] = 4000
    pool = Pool(g, B, 4000, 128, seed=9).fill(lens, 10).to_device()
    q = bf16_normal((B, 2, hd), 11)
    out = f64(decode_gpu(g, pool, q, lens))
    for b in [*range(0, B, 9), B // 3 - 1, B // 3, B // 3 + 1, B - 1]:
        heads = [K.read_rows(pool.data, pool.table[b], h, range(lens[b]), 128) for h in (0, 1)]
        kk, vv = (np.stack([h[i] for h in heads])[None] for i in (0, 1))
        ref, mag = attention_and_scale(f64(q)[b:b + 1, None], kk, vv, lens[b:b + 1, None] - 1, lens[b:b + 1], 2, g)
        assert_within(out[b:b + 1], ref[:, 0], mag[:, 0], C_DECODE, f"sequence {b}", keys=lens[b])


@pytest.mark.parametrize("B,window", [(300, 0), (700, 20)])
def test_decode_many_sequences(B, window):
    """More sequences than a CTA has threads."""
    g = geometry(W.SLIDING if window else W.FULL, 64, H=2, Hkv=1, window=window)
    lens = np.random.default_rng(B).integers(0, 50, B)
    lens[-3:] = 0
    pool = Pool(g, B, 50, 16, seed=6).fill(lens, 7).to_device()
    q = bf16_normal((B, 2, 64), 8)
    out = f64(decode_gpu(g, pool, q, lens))
    k, v = pool.rows(lens, 50)
    ref, mag = attention_and_scale(f64(q)[:, None], k, v, (lens - 1)[:, None], lens, 1, g)
    assert (out[lens == 0] == 0).all()
    assert_within(out, ref[:, 0], mag[:, 0], C_DECODE, keys=50)
