"""Parity of attention with modified scores, of the intervals of keys and of the append with several axes against the
float64 oracles.

Intervals and bf16 stores of the append are exact.  Attention: |error| <= r |out| + c sum_j p_j |v_j|, r the output's
rounding (half a step: bf16 2^-8, float32 2^-24), c twice the relative error d of a weight (numerator and
denominator).  With u = 2^-24, n keys and A the largest sum_d |q_d k_d| + |bias| of the row's keys:
  CUDA cores  scores: hd / 32 products per lane and five shuffled sums, q scaled before and the cap's and bias's
              roundings after, (hd / 32 + 10) u A; a cap's tanh 2^-22 cap; the exponential 2^-21; sums of n terms n u.
  prefill     bf16: weights rounded to bf16, 2^-8 each (so d = 2^-8 + the rest, and c = 2^-7 + ...); the scores' sums of
              hd terms by 16s, (hd / 16 + 10) 2 u A; a cap's tanh 2^-22 of twice the cap in log2 units, 2^-20 cap.
"""

import numpy as np
import pytest

from gemma_dual_geometry_gb300 import build as g4build
from gpu_common import DEV, G, O, W, f64, geometry, params_of, torch
from oracle import mods_oracle as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    g4build.build()
    G.lib()
    yield
    assert G.g4_take_device_error() == 0


def i32(x):
    return torch.tensor(np.ascontiguousarray(x), dtype=torch.int32, device=DEV)


def unit(shape, seed, dtype):
    """Rows of unit mean square, as the append stores them."""
    x = W.normal(shape, seed, W.F32)
    return (x / x.square().mean(-1, keepdim=True).sqrt()).to(W.torch_dtype(dtype))


def ids(rng, B, L, doc, span):
    """Documents and spans of about so many positions, some padding among them."""
    cut = lambda mean: np.cumsum(rng.random((B, L)) < 1.0 / mean, 1)  # noqa: E731
    d, s = cut(doc), cut(span)
    d = np.where(d % 7 == 5, -1 - d, d)
    return d, np.where(s % 2 == rng.integers(0, 2, (B, 1)), s, -1 - s % 3)


# ---------------------------------------------------------------- intervals

@pytest.mark.parametrize("B,T,L,doc,span,window", [
    (1, 1, 1, 1, 1, 0), (3, 1, 50, 7, 3, 4), (2, 100, 100, 20, 10, 0), (5, 333, 1000, 90, 30, 17), (1, 4096, 4096, 500, 90, 64),
    (2, 4097, 4097, 3000, 2000, 512), (3, 2048, 9000, 1, 1, 1), (2, 5000, 12288, 100000, 100000, 700),
    (1, 70000, 70000, 9000, 300, 512), (2, 33, 40001, 20000, 10000, 0), (4, 600, 32768, 3, 5, 2)])
@pytest.mark.parametrize("which", ["both", "docs", "spans", "none"])
def test_visible_ranges(B, T, L, doc, span, window, which):
    rng = np.random.default_rng(L + T + len(which))
    d, s = ids(rng, B, L, doc, span)
    start = rng.integers(0, L - T + 1, B)
    lens = np.minimum(start + rng.integers(0, T + 1, B), L)
    lens[0] = L + 5          # clamped
    if B > 1:
        start[1] = -3        # tokens before the first position
    if B > 2:
        start[2], lens[2] = L - T // 2, L   # tokens past the row's end
    if B > 3:
        lens[3] = 0
    d = d if which in ("both", "docs") else None
    s = s if which in ("both", "spans") else None
    want = M.visible_ranges(window, start, lens, d, s, L, T)
    dd, ds = (None if x is None else i32(x) for x in (d, s))
    for shift in (0, 1):     # outputs 16-byte aligned and not
        out = torch.full((2, B * T + 9), -77, dtype=torch.int32, device=DEV)
        begin, end = out[0, shift:shift + B * T], out[1, shift:shift + B * T]
        G.g4_attn_visible_ranges(window, i32(start), i32(lens), dd, ds, L, B, T, begin, end)
        assert np.array_equal(begin.cpu().numpy(), want[0].ravel()) and np.array_equal(end.cpu().numpy(), want[1].ravel())
        assert (out[:, :shift] == -77).all() and (out[:, shift + B * T:] == -77).all()


def test_visible_ranges_far_starts():
    """Starts far outside of the row give empty intervals."""
    d = i32(np.zeros((5, 10)))
    out = torch.full((2, 5, 4), -1, dtype=torch.int32, device=DEV)
    G.g4_attn_visible_ranges(0, i32([-2 ** 31, 2 ** 31 - 1, 10, -4, 8]), i32([10] * 4 + [-5]), d, None, 10, 5, 4, out[0], out[1])
    assert (out == 0).all()


# ---------------------------------------------------------------- append with axes

GEOS = [(W.SLIDING, 256, 8, 2, 40), (W.FULL, 512, 8, 2, 0), (W.FULL, 128, 8, 1, 0), (W.SLIDING, 64, 3, 3, 17),
        (W.FULL, 256, 4, 2, 0), (W.SLIDING, 512, 4, 4, 33)]


def axes_of(g, n_axes, mixed):
    turns = O.rotated_pairs(g["head_dim"], g["rotary_fraction"])
    return [j % n_axes if mixed else j * n_axes // turns for j in range(turns)]


@pytest.mark.parametrize("geo", GEOS)
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("B,T,n_axes", [(3, 1, 3), (2, 37, 2), (1, 150, 4), (7, 18, 3), (4, 16, 1)])
def test_append_axes(geo, dtype, B, T, n_axes):
    g = geometry(geo[0], geo[1], H=geo[2], Hkv=geo[3], window=geo[4], dtype=dtype)
    hd, H, Hkv, tdt = g["head_dim"], g["n_heads"], g["n_kv_heads"], W.torch_dtype(dtype)
    rng = np.random.default_rng(hd + T)
    ring = geo[0] == W.SLIDING and T == 1
    Lmax = geo[4] if ring else T + 60
    axis = axes_of(g, n_axes, mixed=T % 2 == 0)
    inv = O.rope_inv_freq(hd, g["theta"], g["rotary_fraction"])
    own_freq = n_axes == 2   # frequencies of the caller's own
    if own_freq:
        inv = np.where(inv > 0, (inv * np.float32(0.5)).astype(np.float32), inv)
    pos = rng.integers(-50, 5000, (n_axes, B, T))
    pos[:, :, 0] = pos[:1, :, 0]                  # a token whose axes agree
    if B > 1:
        pos[:, 1] = pos[:, 0]                     # neighbours that share a table
    if n_axes > 1 and B > 2:
        pos[1:, 2], pos[0, 2] = pos[1:, 1], pos[0, 1] + 1   # and that differ in one axis
    pos[0, B - 1, T - 1] = 2 ** 31 - 1
    rows = rng.integers(0, 20, B)[:, None] + np.arange(T)[None] + (1000 if ring else 0)
    if T > 1:
        rows[0, 1], rows[B - 1, T - 1] = -1, Lmax  # not written
    x = {c: W.normal((B, T, h, hd), 50 + i, dtype) for i, (c, h) in enumerate((("q", H), ("k", Hkv), ("v", Hkv)))}
    qw, kw = W.norm_weight(hd, 7), W.norm_weight(hd, 8)
    cache = [torch.full((B, Hkv, Lmax, hd), 3.0, dtype=tdt, device=DEV) for _ in range(2)]
    tab = G.cache_table(2)
    G.set_cache(tab, 0, *cache, g["layer_type"], hd, Hkv, Lmax, B, dtype, ring)
    q = x["q"].to(DEV)
    q_out = torch.empty_like(q)
    axes = G.rope_axes(n_axes, axis, hd, inv if own_freq else None)
    G.g4_kv_append_normrope_axes(params_of(g), tab, 0, axes, q, x["k"].to(DEV), x["v"].to(DEV), qw.to(DEV), kw.to(DEV),
                                 i32(pos), i32(rows), B, T, q_out)
    want = {c: M.normrope_axes(f64(x[c]), f64(w), pos, axis, inv, g["eps"]) for c, w in (("q", qw), ("k", kw))}
    want["v"] = O.rms_norm(f64(x["v"]), None, g["eps"])
    for c in want:
        want[c] = O.store(want[c], dtype)
    kept = [np.full((B, Hkv, Lmax, hd), 3.0) for _ in range(2)]
    for b in range(B):
        for t in range(T):
            if 0 <= rows[b, t] < (Lmax if not ring else 2 ** 31):
                for c, w in zip(kept, (want["k"], want["v"])):
                    c[b, :, rows[b, t] % Lmax] = w[b, t]
    tol = 0 if dtype == W.BF16 else 2e-6 * np.sqrt(hd)   # float32: |y| <= sqrt(hd) w, 2^-20 for norm, rotation, rounding
    for got, ref in ((q_out, want["q"]), (cache[0], kept[0]), (cache[1], kept[1])):
        assert np.abs(f64(got) - ref).max() <= tol
    # a shared layer's q alone, in place
    p = G.layer_params(g["layer_type"], hd, H, Hkv, g["window"], g["theta"], g["rotary_fraction"], g["eps"], 1.0, 0, dtype)
    q2 = q.clone()
    G.g4_kv_append_normrope_axes(p, tab, 1, axes, q2, None, None, qw.to(DEV), None, i32(pos), None, B, T, q2)
    assert torch.equal(q2, q_out)


@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("B,T", [(5, 1), (6, 40), (1, 1100)])
def test_axes_that_agree_store_the_appends_bits(dtype, B, T):
    g = geometry(W.FULL, 256, dtype=dtype)
    Lmax = T + 9
    pos = np.random.default_rng(T).integers(0, 10, B)[:, None] + np.arange(T)[None]
    x = [W.normal((B, T, h, 256), 3 + h, dtype).to(DEV) for h in (8, 2, 2)]
    qw, kw = W.norm_weight(256, 7).to(DEV), W.norm_weight(256, 8).to(DEV)
    got = []
    for call in ("plain", "axes"):
        cache = [torch.zeros((B, 2, Lmax, 256), dtype=x[0].dtype, device=DEV) for _ in range(2)]
        tab = G.cache_table(1)
        G.set_cache(tab, 0, *cache, W.FULL, 256, 2, Lmax, B, dtype)
        out = torch.empty_like(x[0])
        if call == "plain":
            G.g4_kv_append_normrope(params_of(g), tab, 0, *x, qw, kw, i32(pos), B, T, out)
        else:
            G.g4_kv_append_normrope_axes(params_of(g), tab, 0, G.rope_axes(3, axes_of(g, 3, True), 256), *x, qw, kw,
                                         i32(np.stack([pos] * 3)), i32(pos), B, T, out)
        got.append([out, *cache])
    assert all(torch.equal(a, b) for a, b in zip(*got))


# ---------------------------------------------------------------- attention

SLOPES = lambda H: 2.0 ** (-8.0 * np.arange(1, H + 1) / H)  # noqa: E731


def check(got, want, mass, size, g, n, cap, tensor_cores, what):
    A = size[..., None]
    hd = g["head_dim"]
    if tensor_cores:
        d = 2.0 ** -8 + (hd / 16 + 10) * 2 * U * A + 2.0 ** -20 * cap + 2.0 ** -21 + n * U
    else:
        d = (hd / 32 + 10) * U * A + 2.0 ** -22 * cap + 2.0 ** -21 + n * U
    r = 2.0 ** -8 if g["dtype"] == W.BF16 else U
    bound = r * np.abs(want) + 2 * d * mass + 1e-30
    err = np.abs(got - want)
    assert np.isfinite(got).all(), what
    assert (err <= bound).all(), f"{what}: {(err / bound).max():.2f} of the bound at {np.unravel_index((err / bound).argmax(), err.shape)}"


class Case:
    """A cache of B sequences of `lens` positions (rows past them NaN; a ring's rows all written)."""

    def __init__(self, geo, lens, Lmax, dtype, seed, ring=False):
        self.g = geometry(geo[0], geo[1], H=geo[2], Hkv=geo[3], window=geo[4], dtype=dtype)
        self.lens, self.Lmax, self.ring, self.dtype = np.asarray(lens), Lmax, ring, dtype
        B, hd, Hkv = len(lens), geo[1], geo[3]
        self.k, self.v = unit((B, Hkv, Lmax, hd), seed, dtype), unit((B, Hkv, Lmax, hd), seed + 1, dtype)
        if not ring:
            for b, n in enumerate(lens):
                self.k[b, :, n:] = float("nan")
                self.v[b, :, n:] = float("nan")
        self.dk, self.dv = self.k.to(DEV), self.v.to(DEV)
        self.table = G.cache_table(1)
        G.set_cache(self.table, 0, self.dk, self.dv, geo[0], hd, Hkv, Lmax, B, dtype, ring)
        self.params = params_of(self.g)

    def reference(self, q, q_pos, begin, end, held, cap, slopes):
        """Oracle rows of q [B, T, H, hd]; sequence b holds positions up to held[b]."""
        B, T, H, hd = q.shape
        group = H // self.g["n_kv_heads"]
        out, mass, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3])
        k, v = f64(self.k), f64(self.v)
        for b in range(B):
            at, rows = O.key_rows(int(held[b]), self.Lmax, self.ring)
            for h in range(H):
                out[b, :, h], mass[b, :, h], size[b, :, h] = M.attention_rows(
                    q[b, :, h], k[b, h // group, rows], v[b, h // group, rows], at, q_pos[b], begin[b], end[b], cap,
                    0.0 if slopes is None else slopes[h])
        return out, mass, size


def run_prefill(geo, start, T, Lmax, mask, cap, bias, dtype=W.BF16, seed=1, ring=False, doc=60, span=25):
    B = len(start)
    start = np.asarray(start)
    rng = np.random.default_rng(seed)
    lens = start + T if mask == "causal" else np.minimum(start + rng.integers(1, T + 1, B), Lmax)
    c = Case(geo, lens, Lmax, dtype, seed, ring)
    q = unit((B, T, geo[2], geo[1]), seed + 2, dtype)
    at = start[:, None] + np.arange(T)[None]
    begin, end = M.default_intervals(at, geo[0], geo[4])
    given = (None, None)
    if mask != "causal":
        d, s = ids(rng, B, Lmax, doc, span)
        begin, end = M.visible_ranges(geo[4], start, lens, d if mask != "spans" else None, s if mask != "docs" else None,
                                      Lmax, T)
        given = (i32(begin), i32(end))
    slopes = SLOPES(geo[2]) if bias else None
    mods = G.score_mods(cap, None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device=DEV), *given)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=DEV)
    G.g4_attn_prefill_mods(c.params, c.table, 0, mods, q.to(DEV), i32(start), B, T, out)
    want, mass, size = c.reference(f64(q), at, begin, end, lens, cap, slopes)
    check(f64(out), want, mass, size, c.g, int(lens.max()), cap, dtype == W.BF16, (geo, start, T, mask, cap, bias))
    empty = np.asarray(begin) >= np.asarray(end)
    assert (f64(out)[empty] == 0).all()
    return empty.any()


@pytest.mark.parametrize("geo", GEOS)
@pytest.mark.parametrize("mask", ["causal", "docs", "spans", "both"])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (50.0, False), (0.0, True), (20.0, True)])
def test_prefill_mods(geo, mask, cap, bias):
    run_prefill(geo, [0, 130, 7], 150, 300, mask, cap, bias, seed=geo[1] + len(mask))


@pytest.mark.parametrize("geo", GEOS)
@pytest.mark.parametrize("start,T,Lmax", [([0], 1, 1), ([5], 1, 200), ([0, 3], 2, 9), ([0], 127, 127), ([1], 128, 129),
                                          ([0, 127], 129, 256), ([0, 500], 385, 900)])
def test_prefill_mods_lengths(geo, start, T, Lmax):
    run_prefill(geo, start, T, Lmax, "both", 30.0, False, seed=T)
    run_prefill(geo, start, T, Lmax, "causal", 5.0, True, seed=T + 1)


@pytest.mark.parametrize("geo", [GEOS[0], GEOS[3], GEOS[4]])
@pytest.mark.parametrize("mask,cap,bias", [("causal", 0.0, False), ("both", 50.0, True), ("spans", 0.0, True), ("docs", 8.0, False)])
def test_prefill_mods_float32(geo, mask, cap, bias):
    run_prefill(geo, [0, 40, 11], 90, 170, mask, cap, bias, dtype=W.F32, seed=5)


@pytest.mark.parametrize("geo,rows", [(GEOS[0], 256), (GEOS[3], 128), (GEOS[5], 384)])
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
def test_prefill_mods_ring(geo, rows, dtype):
    run_prefill(geo, [0, 1000, 77], 80, rows, "causal", 50.0, True, dtype=dtype, seed=9, ring=True)


@pytest.mark.parametrize("cap", [2.0 ** -10, 0.5, 1024.0])
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
def test_prefill_mods_extreme_caps(cap, dtype):
    run_prefill(GEOS[4], [0, 20], 100, 150, "docs", cap, False, dtype=dtype, seed=3)


def test_prefill_mods_many_items():
    """More work items than SMs, of very different sizes, and rows that see nothing."""
    assert run_prefill((W.SLIDING, 64, 8, 2, 100), [0, 30, 200, 64], 700, 1000, "both", 50.0, False, seed=4, doc=300, span=90)
    run_prefill((W.FULL, 128, 8, 4, 0), [0, 100], 1500, 1600, "docs", 0.0, True, seed=6, doc=400)


def run_decode(geo, lens, Lmax, cap, bias, begin=None, dtype=W.BF16, seed=1, ring=False, most=None):
    B = len(lens)
    lens = np.asarray(lens)
    c = Case(geo, lens, Lmax, dtype, seed, ring)
    q = unit((B, geo[2], geo[1]), seed + 2, dtype)
    slopes = SLOPES(geo[2]) if bias else None
    mods = G.score_mods(cap, None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device=DEV),
                        None if begin is None else i32(begin))
    most = most or max(1, int(lens.max()))
    size = G.g4_attn_decode_mods_workspace_size(c.params, B, most)
    ws = torch.zeros(max(16, size), dtype=torch.uint8, device=DEV)
    outs = []
    for _ in range(2):   # the workspace serves again
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=DEV)
        G.g4_attn_decode_mods(c.params, c.table, 0, mods, q.to(DEV), i32(lens), B, most, out, ws, size)
        outs.append(out)
    assert torch.equal(*outs)
    at = (lens - 1)[:, None]
    lo, hi = M.default_intervals(at, geo[0], geo[4])
    if begin is not None:
        lo = np.maximum(lo, np.asarray(begin)[:, None])
    want, mass, mag = c.reference(f64(q)[:, None], at, lo, hi, lens, cap, slopes)
    check(f64(outs[0])[:, None], want, mass, mag, c.g, int(lens.max()), cap, False, (geo, lens, cap, bias))
    assert (f64(outs[0])[(lo >= hi)[:, 0]] == 0).all()


@pytest.mark.parametrize("geo", GEOS)
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (50.0, False), (0.0, True), (20.0, True)])
def test_decode_mods(geo, dtype, cap, bias):
    run_decode(geo, [1, 300, 0, 77, 64], 310, cap, bias, dtype=dtype, seed=geo[1])
    run_decode(geo, [1, 300, 0, 77, 64], 310, cap, bias, begin=[0, 290, 0, 77, 63], dtype=dtype, seed=geo[1], most=310)


@pytest.mark.parametrize("geo,lens", [(GEOS[1], [5000]), (GEOS[2], [3000, 1, 2999, 40]), (GEOS[4], [700] * 70),
                                      ((W.SLIDING, 256, 8, 2, 512), [600, 511, 512, 513, 2000]), (GEOS[0], [900] * 90)])
def test_decode_mods_splits(geo, lens):
    run_decode(geo, lens, max(lens), 50.0, True, seed=7)
    run_decode(geo, lens, max(lens), 0.0, True, begin=np.asarray(lens) * 2 // 3, seed=8)


def test_decode_mods_ring():
    run_decode((W.SLIDING, 256, 8, 2, 64), [1, 63, 64, 65, 1000, 100000], 64, 50.0, True, ring=True, seed=3)
    run_decode((W.SLIDING, 64, 4, 4, 200), [500, 90, 2 ** 31 - 1], 200, 0.0, True, begin=[400, 95, 0], ring=True, seed=4)


def test_intervals_reach_any_key():
    """Intervals that leave the causal order (keys behind the query), that are reversed, or that pass the cache's ends."""
    geo, T, L = (W.SLIDING, 128, 4, 2, 8), 140, 300
    rng = np.random.default_rng(0)
    c = Case(geo, [L], L, W.BF16, 3)
    q = unit((1, T, 4, 128), 5, W.BF16)
    begin, end = rng.integers(-20, L, (1, T)), rng.integers(0, L + 50, (1, T))
    begin[0, :3], end[0, :3] = [-2 ** 31, 2 ** 31 - 1, 0], [2 ** 31 - 1, -2 ** 31, 0]
    out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    G.g4_attn_prefill_mods(c.params, c.table, 0, G.score_mods(0.0, None, i32(begin), i32(end)), q.to(DEV), i32([160]), 1, T, out)
    want, mass, size = c.reference(f64(q), 160 + np.arange(T)[None], begin, end, [L], 0.0, None)
    check(f64(out), want, mass, size, c.g, L, 0.0, True, "any")
    assert (f64(out)[begin >= end] == 0).all()
