"""The paged 4-bit cache where its callers go past the plain run of things: tables whose blocks were taken away,
rows that hold no numbers, prompt-sized batches.  Bytes, ids and lengths are exact."""

import numpy as np
import pytest

from gemma_dual_geometry_gb300 import build as g4build

from kv4_common import (DEV, G, K, O, Pool, W, assert_within, attention_and_scale, bf16_normal, f64, geometry, i32,
                        params_of, torch)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    g4build.build()
    G.lib()
    yield
    assert G.g4_take_device_error() == 0


# ---------------------------------------------------------------- block assignment

@pytest.mark.parametrize("B,T,bs,width,gone", [(1, 1, 16, 5, "some"), (6, 3, 16, 40, "some"), (64, 1, 64, 130, "front"),
                                               (64, 5, 16, 300, "some"), (96, 2048, 16, 130, "front"), (9, 4, 32, 20, "all"),
                                               (700, 3, 16, 70, "some"), (700, 3, 16, 70, "front"), (130, 1, 16, 3, "all")])
@pytest.mark.parametrize("short", [False, True])
@pytest.mark.parametrize("alias", [False, True])
def test_assign_gives_back_only_blocks_of_the_pool(B, T, bs, width, gone, short, alias):
    """Entries that hold no block (a caller took it away: those before a window, or any) are not put on the free
    list when their sequence shrinks or ends; all that does go there, and who is served from it, stays exact."""
    rng = np.random.default_rng(B * 7 + T + len(gone))
    n = B * width + 9
    lens = rng.integers(0, width * bs + 1, B)
    lens[0] = width * bs
    table = np.full((B, width), -1)
    order = rng.permutation(n)
    at = 0
    for b in range(B):
        have = -(-int(lens[b]) // bs)
        ids = order[at:at + have].copy()
        at += have
        if gone == "all":
            away = np.ones(have, bool)
        elif gone == "front":
            away = np.arange(have) < have - 2
        else:
            away = rng.random(have) < 0.3
        ids[away] = rng.choice([-1, n, n + 7, -2 ** 31, 2 ** 31 - 1], int(away.sum()))
        table[b, :have] = ids
    free = np.full(n, -1)
    count = min(3, n - at) if short else n - at
    free[:count] = order[at:at + count]
    kind = rng.random(B)
    new = np.where(kind < 0.4, 0, np.where(kind < 0.6, lens // 2, lens + rng.integers(0, T + 1, B)))
    new[0] = 0
    want = K.assign_blocks(lens, new, T, bs, n, free, count, table)
    assert all(0 <= x < n for x in want[1][:want[2]])
    d_old, d_new, d_free, d_count, d_table = i32(lens), i32(new), i32(free), i32([count]), i32(table)
    out = d_old if alias else i32(np.zeros(B))
    left = d_count if alias else i32([0])
    pos, slots = i32(np.zeros((B, T))), i32(np.zeros((B, T)))
    for _ in range(1 if alias else 2):   # a repeated call repeats its results
        G.g4_kv4_assign_blocks(B, T, bs, n, width, d_old, d_new, d_free, d_count, d_table, out, left, pos, slots)
    got = [x.cpu().numpy().ravel() for x in (d_table, d_free, left, out, pos, slots)]
    got[1], want = got[1][:want[2]], list(want)
    want[1] = want[1][:want[2]]          # (what lies behind the count is nobody's)
    for name, g, w in zip(("table", "free", "count", "lens", "positions", "slots"), got, want):
        assert np.array_equal(g, np.asarray(w).ravel()), name


# ---------------------------------------------------------------- append

def store(data, slots, k, v, block_size, k_exp=0):
    """Rows k, v [N, Hkv, hd] (bf16 values) into data at slots [N] >= 0, by the oracle."""
    kc, ks, vc, vs = K.record_offsets(k.shape[-1])
    (kq, ksc), (vq, vsc) = K.quantise(k, k_exp), K.quantise(v)
    at = np.arange(k.shape[1])[None, :, None]
    block, group, m = (slots // block_size)[:, None, None], (slots % block_size // 16)[:, None, None], slots % 16
    for code, scale, co, so in ((kq, ksc, kc, ks), (vq, vsc, vc, vs)):
        data[block, at, group, co[m][:, None, 0::2]] = code[..., 0::2] | code[..., 1::2] << 4
        data[block, at, group, so[m][:, None, 0::16]] = scale


@pytest.mark.parametrize("geo", [(W.SLIDING, 64, 3, 3, 17), (W.FULL, 128, 8, 1, 0), (W.SLIDING, 256, 8, 2, 40),
                                 (W.FULL, 512, 4, 2, 0)])
@pytest.mark.parametrize("B,T", [(5, 520), (7, 520), (8, 515), (1, 1030)])
def test_append_bytes_of_prompts(geo, B, T):
    """From 1024 CTAs on a CTA takes all rows of its tokens: groups of four tokens, and a remainder of one or three."""
    g = geometry(geo[0], geo[1], H=geo[2], Hkv=geo[3], window=geo[4])
    hd, H, Hkv, bs = g["head_dim"], g["n_heads"], g["n_kv_heads"], 64
    rng = np.random.default_rng(hd + B)
    start = rng.integers(0, 300, B)
    start[1:3] = start[0]           # neighbours whose positions agree
    pool = Pool(g, B, 300 + T, bs, seed=hd + B)
    x = {c: bf16_normal((B, T, h, hd), 70 + i) for i, (c, h) in enumerate((("q", H), ("k", Hkv), ("v", Hkv)))}
    qw, kw = W.norm_weight(hd, 7), W.norm_weight(hd, 8)
    pos = start[:, None] + np.arange(T)[None, :]
    slots = np.take_along_axis(pool.table, pos // bs, 1) * bs + pos % bs
    slots[rng.random((B, T)) < 0.1] = -1
    slots[B - 1, T - 3:] = pool.n * bs   # outside the pool
    pool.to_device()
    q = x["q"].to(DEV)
    q_out = torch.empty_like(q)
    G.g4_kv4_append_normrope(params_of(g), pool.pools, 0, q, x["k"].to(DEV), x["v"].to(DEV), qw.to(DEV), kw.to(DEV),
                             i32(pos), i32(slots), B, T, q_out)
    kn, vn = O.normrope_kv(f64(x["k"]), f64(x["v"]), f64(kw), pos, hd, g["theta"], g["rotary_fraction"], g["eps"])
    there = (slots >= 0) & (slots < pool.n * bs)
    want = pool.data.copy()
    store(want, slots[there], O.round_bf16(kn)[there], O.round_bf16(vn)[there], bs)
    got = pool.d.cpu().numpy()
    assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ"
    ref_q = O.round_bf16(O.normrope_q(f64(x["q"]), f64(qw), pos, hd, g["theta"], g["rotary_fraction"], g["eps"]))
    assert np.array_equal(f64(q_out), ref_q)
    # a layer that reads the pool of another: q alone, the pool left as it was
    pools = G.kv4_pool_table(2)
    pools[0] = pool.pools[0]
    again = torch.empty_like(q)
    G.g4_kv4_append_normrope(params_of(g, src=0), pools, 1, q, None, None, qw.to(DEV), None, i32(pos), None, B, T, again)
    assert torch.equal(again, q_out) and np.array_equal(pool.d.cpu().numpy(), want)


@pytest.mark.parametrize("geo", [(W.SLIDING, 64, 3, 3, 17), (W.FULL, 128, 8, 1, 0), (W.SLIDING, 256, 8, 2, 40),
                                 (W.FULL, 512, 4, 2, 0)])
def test_append_bytes_of_blocks_without_numbers(geo):
    """A 16 that holds a NaN or an infinity: scale NaN and codes 0, the other 16s of its row as ever."""
    g = geometry(geo[0], geo[1], H=geo[2], Hkv=geo[3], window=geo[4])
    hd, H, Hkv, T, bs = g["head_dim"], g["n_heads"], g["n_kv_heads"], 3, 16
    pool = Pool(g, 1, T, bs, seed=1)
    q, k, v = (bf16_normal((1, T, h, hd), s) for h, s in ((H, 1), (Hkv, 2), (Hkv, 3)))
    kw = W.norm_weight(hd, 4)
    kw[20], kw[40] = float("nan"), float("inf")   # elements of k (and what RoPE turns with them)
    v[0, 1, 0, 9] = float("nan")                  # a whole row of v
    pos = np.arange(T)[None]
    slots = np.array([[pool.slot(0, p) for p in range(T)]])
    pool.to_device()
    G.g4_kv4_append_normrope(params_of(g), pool.pools, 0, q.to(DEV), k.to(DEV), v.to(DEV), W.norm_weight(hd, 5).to(DEV),
                             kw.to(DEV), i32(pos), i32(slots), 1, T, torch.empty_like(q, device=DEV))
    with np.errstate(invalid="ignore"):
        kn, vn = O.normrope_kv(f64(k), f64(v), f64(kw), pos, hd, g["theta"], g["rotary_fraction"], g["eps"])
    # pairs past the rotated ones pass through as they are (the oracle adds 0 times the other element: NaN next to an infinity)
    still = np.arange(hd) % (hd // 2) >= O.rotated_pairs(hd, g["rotary_fraction"])
    kn[..., still] = O.rms_norm(f64(k), f64(kw), g["eps"])[..., still]
    assert np.isnan(vn[0, 1, 0]).all() and np.isfinite(kn).any() and not np.isfinite(kn[..., 20]).any()
    want = pool.data.copy()
    store(want, slots[0], O.round_bf16(kn)[0], O.round_bf16(vn)[0], bs)
    got = pool.d.cpu().numpy()
    assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ"


# ---------------------------------------------------------------- as they are used

def test_blocks_behind_a_window_are_taken_away():
    """A sliding layer with a table of its own, whose caller takes blocks back as they fall behind the window: the
    pool is a fraction of the contexts it serves, attention is that over all positions, prompts and steps alike,
    and once the sequences have ended the free list holds every block once."""
    window, bs, hd, H, Hkv, B, n = 20, 16, 64, 4, 2, 3, 15
    g = geometry(W.SLIDING, hd, H=H, Hkv=Hkv, window=window)
    p = params_of(g)
    width = 12                                                     # 36 blocks' worth of positions, 15 blocks
    pools = G.kv4_pool_table(1)
    data = torch.full((G.kv4_pool_bytes(n, Hkv, bs, hd),), 255, dtype=torch.uint8, device=DEV)
    G.set_kv4_pool(pools, 0, data, W.SLIDING, hd, Hkv, n, bs)
    table, free, count = i32(np.full((B, width), -1)), i32(np.arange(n)), i32([n])
    lens = i32(np.zeros(B))
    qw, kw = W.norm_weight(hd, 1).to(DEV), W.norm_weight(hd, 2).to(DEV)
    most = width * bs
    rows = [[] for _ in range(B)]
    held = np.zeros(B, int)
    plan = [(40, [40, 17, 33])] + [(30, [40 + 30 * i, 17 + 25 * i, 33 + 14 * i]) for i in range(1, 4)]
    plan += [(1, [130 + i, 92 + i, 75 + i]) for i in range(1, 25)] + [(1, [0, 0, 0])]
    for step, (T, want) in enumerate(plan):
        pos, slots, start = i32(np.zeros((B, T))), i32(np.zeros((B, T))), lens.clone()
        G.g4_kv4_assign_blocks(B, T, bs, n, width, lens, i32(want), free, count, table, lens, count, pos, slots)
        assert lens.tolist() == want, step
        if not any(want):
            break
        q, k, v = (bf16_normal((B, T, h, hd), 10 * step + i) for i, h in enumerate((H, Hkv, Hkv)))
        qo = torch.empty_like(q, device=DEV)
        out = torch.empty_like(qo)
        G.g4_kv4_append_normrope(p, pools, 0, q.to(DEV), k.to(DEV), v.to(DEV), qw, kw, pos, slots, B, T, qo)
        if T == 1:
            nb = G.g4_kv4_decode_workspace_size(p, B, most)
            ws = torch.zeros(max(16, nb), dtype=torch.uint8, device=DEV)
            G.g4_kv4_attn_decode(p, pools, 0, qo, table, width, lens, B, most, out, ws, nb)
        else:
            nb = G.g4_kv4_prefill_workspace_size(p, B, T, most)
            ws = torch.full((nb,), 255, dtype=torch.uint8, device=DEV)
            G.g4_kv4_attn_prefill(p, pools, 0, qo, table, width, start, lens, B, T, most, out, ws, nb)
        at = pos.cpu().numpy()
        qn = O.round_bf16(O.normrope_q(f64(q), f64(qw), at, hd, g["theta"], 1.0, g["eps"]))
        kn, vn = O.normrope_kv(f64(k), f64(v), f64(kw), at, hd, g["theta"], 1.0, g["eps"])
        kn, vn = (K.values(*K.quantise(O.round_bf16(x))) for x in (kn, vn))
        for b in range(B):
            fresh = want[b] - held[b]
            rows[b] += [(kn[b, t], vn[b, t]) for t in range(fresh)]
            kk, vv = (np.stack([r[i] for r in rows[b]], 1)[None] for i in (0, 1))
            ref, mag = attention_and_scale(qn[b:b + 1, :fresh], kk, vv, held[b] + np.arange(fresh)[None],
                                           np.array([want[b]]), Hkv, g)
            assert_within(f64(out[b:b + 1, :fresh]), ref, mag, 2.0 ** -8 if T == 1 else 2.0 ** -7, f"step {step}",
                          keys=window if T == 1 else 0)   # (the bounds of test_gpu_kv4)
        held = np.array(want)
        # the next token sees the positions from want - window + 1 on: blocks wholly before that go back
        ids, stack = table.cpu().numpy(), free.cpu().numpy()[:count.item()].tolist()
        for b in range(B):
            for e in range(max(0, want[b] - window + 1) // bs):
                if ids[b, e] >= 0:
                    stack.append(int(ids[b, e]))
                    ids[b, e] = -1
        table.copy_(i32(ids))
        free[:len(stack)] = i32(stack)
        count.fill_(len(stack))
    assert count.item() == n and sorted(free.tolist()) == list(range(n))
