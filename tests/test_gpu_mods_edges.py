"""Modified scores, intervals and several axes where their callers go past the plain run of things: all of them in a
stack's run, captured graphs, other streams, NaN and infinities in places that are masked, workspaces in turn."""

import numpy as np
import pytest

from gemma_dual_geometry_gb300 import build as g4build
from gemma_dual_geometry_gb300.stack import AttnStack
from gpu_common import DEV, G, O, W, f64, params_of, torch
from oracle import mods_oracle as M
from test_gpu_mods import GEOS, SLOPES, Case, axes_of, check, geometry, i32, ids, unit

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    g4build.build()
    G.lib()
    yield
    assert G.g4_take_device_error() == 0


# ---------------------------------------------------------------- NaN and infinities in masked places

@pytest.mark.parametrize("geo", GEOS)
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (50.0, True)])
def test_prefill_keeps_nan_to_those_who_see_it(geo, dtype, cap, bias):
    """Three documents of a row: NaN and infinities in the second one's keys and values leave the others' outputs as they
    were (but for a rounding) and reach the second one's queries that see them."""
    T = 300
    c = Case(geo, [T], T, dtype, 5)
    doc = np.repeat([0, 1, 2], [110, 70, 120])[None]
    begin, end = M.visible_ranges(0, [0], [T], doc, None, T, T)   # (no window: the document's later tokens see all)
    q = unit((1, T, geo[2], geo[1]), 9, dtype).to(DEV)
    slopes = torch.tensor(SLOPES(geo[2]), dtype=torch.float32, device=DEV) if bias else None
    mods = G.score_mods(cap, slopes, i32(begin), i32(end))

    def run():
        out = torch.empty_like(q)
        G.g4_attn_prefill_mods(c.params, c.table, 0, mods, q, i32([0]), 1, T, out)
        return f64(out)[0]

    clean = run()
    for bad in (float("nan"), float("inf"), float("-inf")):
        for k_too in (False, True):
            saved = c.dk.clone(), c.dv.clone()
            c.dv[0, :, 120, ::7] = bad
            if k_too:
                c.dk[0, :, 125, 3] = bad
            got = run()
            for s in (slice(0, 120), slice(180, 300)):   # (of the second document: what lies before)
                if dtype == W.F32:
                    assert np.array_equal(got[s], clean[s])
                else:   # (rows formed again: each is off by 2^-7 of the mass and a rounding of 2^-8 at most)
                    assert np.isfinite(got[s]).all()
                    assert np.abs(got[s] - clean[s]).max() <= 2.0 ** -5 * np.abs(f64(c.v)).max()
            assert not np.isfinite(got[120:180, :, 0]).any()
            c.dk.copy_(saved[0])
            c.dv.copy_(saved[1])
    assert np.array_equal(run(), clean)


@pytest.mark.parametrize("geo", [GEOS[0], GEOS[1], GEOS[2], GEOS[3], GEOS[5]])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, True)])
def test_prefill_rows_formed_again_are_right(geo, cap, bias):
    """NaN and infinities in values that some of a tile's queries see: the others' rows against the oracle."""
    T, L = 200, 330
    c = Case(geo, [L], L, W.BF16, 6)
    begin, end = np.full((1, T), 40), 41 + np.arange(T)[None] // 2
    slopes = SLOPES(geo[2]) if bias else None
    c.dv[0, :, 30:40] = float("nan")
    c.dv[0, :, 100] = float("nan")
    c.dv[0, :, 103] = float("inf")
    c.dv[0, :, 145:] = float("inf")
    c.dk[0, :, 150:] = float("nan")
    q = unit((1, T, geo[2], geo[1]), 9, W.BF16)
    out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    d_slopes = torch.tensor(slopes, dtype=torch.float32, device=DEV) if bias else None
    G.g4_attn_prefill_mods(c.params, c.table, 0, G.score_mods(cap, d_slopes, i32(begin), i32(end)), q.to(DEV), i32([130]), 1, T,
                           out)
    want, mass, size = c.reference(f64(q), 130 + np.arange(T)[None], begin, end, [145], cap, slopes)
    clean = end[0] <= 100
    check(f64(out)[:, clean], want[:, clean], mass[:, clean], size[:, clean], c.g, L, cap, True, geo)
    assert np.isnan(f64(out)[:, ~clean]).all()


@pytest.mark.parametrize("geo", GEOS)
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
def test_prefill_rows_that_see_nothing_are_zero(geo, dtype):
    """Empty intervals (of all kinds) among rows that see NaN and infinities, of queries that are NaN themselves."""
    T = 140
    c = Case(geo, [T], T, dtype, 4)
    c.dv[0, :, 10] = float("nan")
    c.dv[0, :, 20] = float("-inf")
    c.dk[0, :, 30] = float("inf")
    q = unit((1, T, geo[2], geo[1]), 2, dtype).to(DEV)
    begin, end = np.zeros((1, T), int), np.full((1, T), 60)
    empty = np.arange(T) % 3 == 0
    begin[0, empty] = np.resize([0, 60, 500, 2 ** 31 - 1, 50, -3, 0, -2 ** 31, 2 ** 31 - 1], empty.sum())
    end[0, empty] = np.resize([0, 60, 3, -2 ** 31, 40, -3, -2 ** 31, -2 ** 31 + 1, 2 ** 31 - 1], empty.sum())
    q[0, 3] = float("nan")
    out = torch.empty_like(q)
    G.g4_attn_prefill_mods(c.params, c.table, 0, G.score_mods(0.0, None, i32(begin), i32(end)), q, i32([0]), 1, T, out)
    assert (f64(out)[0, empty] == 0).all() and np.isnan(f64(out)[0, ~empty]).all()


@pytest.mark.parametrize("n", [32768, 32769])
def test_prefill_rows_too_long_to_form_again(n):
    """Rows of up to 2^15 keys are formed again, longer ones are NaN, as documented; other tiles are as they were."""
    geo, T = (W.FULL, 64, 2, 1, 0), 256
    c = Case(geo, [n + 200], n + 200, W.BF16, 7)
    c.dv[:, :, n + 1] = float("nan")
    q = unit((1, T, 2, 64), 8, W.BF16)
    begin, end = np.full((1, T), 1), np.full((1, T), n + 1)
    end[0, :100] = n + 2   # (the first tile's only)
    begin[0, :100] = n + 1
    out = torch.empty_like(q, device=DEV)
    mods = G.score_mods(0.0, None, i32(begin), i32(end))
    G.g4_attn_prefill_mods(c.params, c.table, 0, mods, q.to(DEV), i32([n - 100]), 1, T, out)
    got = f64(out)
    assert np.isnan(got[0, :100]).all() and np.isnan(got[0, 100:128]).all() == (n > 32768)
    some = [100, 127, 128, 255] if n <= 32768 else [128, 255]
    c.v[:, :, n + 1] = 0.0
    at = (n - 100 + np.arange(T))[None, some]
    want, mass, size = c.reference(f64(q)[:, some], at, begin[:, some], end[:, some], [n + 200], 0.0, None)
    check(got[:, some], want, mass, size, c.g, n, 0.0, True, n)


@pytest.mark.parametrize("geo,lens", [(GEOS[0], [100, 300]), (GEOS[1], [300, 90]), (GEOS[2], [700, 260]),
                                      (GEOS[3], [30, 200])])
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
def test_decode_keeps_to_its_keys(geo, lens, dtype):
    """NaN in all rows before a sequence's first key and behind its last."""
    c = Case(geo, lens, max(lens) + 70, dtype, 8)
    begin = [n // 3 for n in lens]
    for b, n in enumerate(begin):
        c.k[b, :, :n] = float("nan")
        c.v[b, :, :n] = float("inf")
    c.dk.copy_(c.k.to(DEV))
    c.dv.copy_(c.v.to(DEV))
    q = unit((2, geo[2], geo[1]), 3, dtype)
    most = max(lens) + 70
    size = G.g4_attn_decode_mods_workspace_size(c.params, 2, most)
    ws = torch.zeros(max(16, size), dtype=torch.uint8, device=DEV)
    out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    mods = G.score_mods(50.0, None, i32(begin))
    G.g4_attn_decode_mods(c.params, c.table, 0, mods, q.to(DEV), i32(lens), 2, most, out, ws, size)
    at = np.asarray(lens)[:, None] - 1
    lo, hi = M.default_intervals(at, geo[0], geo[4])
    want, mass, mag = c.reference(f64(q)[:, None], at, np.maximum(lo, np.asarray(begin)[:, None]), hi, lens, 50.0, None)
    check(f64(out)[:, None], want, mass, mag, c.g, max(lens), 50.0, False, geo)


@pytest.mark.parametrize("geo", [GEOS[0], GEOS[1], GEOS[3]])
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("n", [70, 300, 900])
def test_decode_keeps_visible_nan(geo, dtype, n):
    """Scores that are NaN for one key, for a run of keys and for all: so is the row."""
    c = Case(geo, [n], n, dtype, 8)
    q = unit((1, geo[2], geo[1]), 3, dtype).to(DEV)
    size = G.g4_attn_decode_mods_workspace_size(c.params, 1, n)
    ws = torch.zeros(max(16, size), dtype=torch.uint8, device=DEV)
    for lo, hi in ((n - 2, n - 1), (n - 17, n - 1), (n - 1, n), (0, n)):
        c.dk.copy_(c.k)
        c.dk[0, :, lo:hi] = float("nan")
        for mods in (None, G.score_mods(30.0)):
            out = torch.empty_like(q)
            G.g4_attn_decode_mods(c.params, c.table, 0, mods, q, i32([n]), 1, n, out, ws, size)
            assert torch.isnan(out).all()
            out = torch.empty_like(q)
            G.g4_attn_prefill_mods(c.params, c.table, 0, mods, q.view(1, 1, geo[2], geo[1]), i32([n - 1]), 1, 1, out)
            assert torch.isnan(out).all()


# ---------------------------------------------------------------- a run of them together

CFG = dict(B=3, H=8, Hkv=2, dtype=W.BF16, seed=77, types=[W.SLIDING, W.FULL, W.SLIDING, W.FULL], n_shared=2,
           geom={W.SLIDING: dict(head_dim=64, theta=1e4, rotary_fraction=1.0, window=40),
                 W.FULL: dict(head_dim=128, theta=1e6, rotary_fraction=0.25, window=0)})


@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("side_stream", [False, True])
def test_a_prompt_with_images_and_its_answer(dtype, side_stream):
    """A padded batch of prompts with images, packed documents and capped scores through a stack of owning and shared
    layers: intervals, appends with three axes, prefill; then steps of a new token each: append, decode."""
    cfg = dict(CFG, dtype=dtype)
    B, T, Lmax, steps, cap = cfg["B"], 170, 190, 3, 40.0
    stream = torch.cuda.Stream() if side_stream else None
    rng = np.random.default_rng(3)
    st = AttnStack(cfg, Lmax, device=DEV, mods=True)
    torch.cuda.synchronize()
    lens = np.array([170, 33, 128])
    doc = np.cumsum(rng.random((B, Lmax)) < 0.02, 1)
    seg = np.cumsum(rng.random((B, Lmax)) < 0.06, 1)
    span = np.where((seg % 2 == 1) & (np.arange(Lmax) < lens[:, None]), seg, -1)
    at = np.arange(T)[None].repeat(B, 0)
    pos = np.stack([at, at // 3, at % 16])
    rows = np.where(at < lens[:, None], at, -1)
    start, d_doc, d_span = i32(np.zeros(B)), i32(doc), i32(span)
    heads = {0: cfg["H"], 1: cfg["Hkv"], 2: cfg["Hkv"]}
    n = len(cfg["types"])
    raw = {(l, s): [W.normal((B, T if s == 0 else 1, heads[i], st.geo[l]["head_dim"]), 1000 * s + 10 * l + i, dtype)
                    for i in range(3)] for l in range(n) for s in range(steps + 1)}
    weights = {l: [W.norm_weight(st.geo[l]["head_dim"], 50 + 2 * l + i) for i in range(2)] for l in range(n)}
    axes_np = {l: axes_of(st.geo[l], 3, l % 2 == 0) for l in range(n)}
    axes = {l: G.rope_axes(3, axes_np[l], st.geo[l]["head_dim"]) for l in range(n)}
    dev = {k: [x.to(DEV) for x in v] for k, v in raw.items()}
    wdev = {l: [x.to(DEV) for x in w] for l, w in weights.items()}
    ranges = {}
    outs, step_outs = {}, {}
    torch.cuda.synchronize()
    with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
        d_lens = i32(lens)
        for lt in (W.SLIDING, W.FULL):
            begin, end = i32(np.zeros((B, T))), i32(np.zeros((B, T)))
            st.visible_ranges(lt, start, d_lens, d_doc, d_span, T, begin, end)
            ranges[lt] = begin, end
        for l in range(n):
            q, k, v = dev[l, 0]
            q_out, out = torch.empty_like(q), torch.empty_like(q)
            st.append_axes(l, axes[l], q, k if st.owns(l) else None, v if st.owns(l) else None, wdev[l][0],
                           wdev[l][1] if st.owns(l) else None, i32(pos), i32(rows), T, q_out)
            st.prefill_attn(l, q_out, start, T, out, mods=G.score_mods(cap, None, *ranges[st.geo[l]["layer_type"]]))
            outs[l] = out
        for s in range(1, steps + 1):
            now = lens + s - 1   # the new token's position
            p = i32(np.stack([now, now // 2, now % 7])[:, :, None])
            d_lens = i32(lens + s)
            begins = {}
            for lt in (W.SLIDING, W.FULL):
                begin, end = i32(np.zeros((B, 1))), i32(np.zeros((B, 1)))
                st.visible_ranges(lt, i32(now), d_lens, d_doc, None, 1, begin, end)
                begins[lt] = begin.view(B)
            for l in range(n):
                q, k, v = dev[l, s]
                q_out, out = torch.empty_like(q), torch.empty((B, cfg["H"], q.shape[3]), dtype=q.dtype, device=DEV)
                st.append_axes(l, axes[l], q, k if st.owns(l) else None, v if st.owns(l) else None, wdev[l][0],
                               wdev[l][1] if st.owns(l) else None, p, i32(now[:, None]), 1, q_out)
                st.decode_attn(l, q_out.view(B, cfg["H"], -1), d_lens, Lmax, out,
                               mods=G.score_mods(cap, None, begins[st.geo[l]["layer_type"]]))
                step_outs[l, s] = out
    torch.cuda.synchronize()

    # the same from the oracle's own rows
    caches = {l: [np.zeros((B, cfg["Hkv"], Lmax, st.geo[l]["head_dim"])) for _ in range(2)]
              for l in range(n) if st.owns(l)}
    inv = {l: O.rope_inv_freq(g["head_dim"], g["theta"], g["rotary_fraction"]) for l, g in enumerate(st.geo)}

    def append(l, s, p, r):
        q, k, v = (f64(x) for x in raw[l, s])
        w = [f64(x) for x in weights[l]]
        if st.owns(l):
            kn = O.store(M.normrope_axes(k, w[1], p, axes_np[l], inv[l], W.EPS), dtype)
            vn = O.store(O.rms_norm(v, None, W.EPS), dtype)
            for b in range(B):
                for t in range(k.shape[1]):
                    if r[b, t] >= 0:
                        caches[l][0][b, :, r[b, t]], caches[l][1][b, :, r[b, t]] = kn[b, t], vn[b, t]
        return O.store(M.normrope_axes(q, w[0], p, axes_np[l], inv[l], W.EPS), dtype)

    def attend(l, q, q_pos, begin, end, held):
        k, v = caches[l if st.owns(l) else st.src[l]]
        group = cfg["H"] // cfg["Hkv"]
        res = [np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3])]
        for b in range(B):
            keys = np.arange(held[b])
            for h in range(cfg["H"]):
                kh, vh = k[b, h // group, :held[b]], v[b, h // group, :held[b]]
                for r, x in zip(res, M.attention_rows(q[b, :, h], kh, vh, keys, q_pos[b], begin[b], end[b], cap)):
                    r[b, :, h] = x
        return res

    # (float32 rows are within 8 x 2^-24 of the oracle's, so that a score of sum |q_d k_d| = A moves by 16 x 2^-24 A: twice
    # what the bound has for float32 sums already; eight times the mass covers it)
    for l in range(n):
        g = dict(st.geo[l], dtype=dtype)
        begin, end = M.visible_ranges(g["window"], np.zeros(B, int), lens, doc, span, Lmax, T)
        for got, want in zip(ranges[g["layer_type"]], (begin, end)):
            assert np.array_equal(got.cpu().numpy(), want)
        want, mass, size = attend(l, append(l, 0, pos, rows), at, begin, end, lens)
        check(f64(outs[l]), want, mass * (1.0 if dtype == W.BF16 else 8.0), size, g, T, cap, dtype == W.BF16, ("prefill", l))
        assert (f64(outs[l])[begin >= end] == 0).all()
    for s in range(1, steps + 1):
        now = (lens + s - 1)[:, None]
        for l in range(n):
            g = dict(st.geo[l], dtype=dtype)
            begin, end = M.visible_ranges(g["window"], now[:, 0], lens + s, doc, None, Lmax, 1)
            p = np.stack([now, now // 2, now % 7])
            want, mass, size = attend(l, append(l, s, p, now), now, begin, end, lens + s)
            check(f64(step_outs[l, s])[:, None], want, mass * (1.0 if dtype == W.BF16 else 8.0), size, g, Lmax,
                  cap, False, ("step", s, l))


# ---------------------------------------------------------------- graphs, streams, workspaces

def test_captured_and_replayed():
    """All four captured into a graph, replayed with other inputs in the same buffers: the eager calls' bits."""
    geo, B, T, L = GEOS[0], 2, 150, 700
    c = Case(geo, [T, T], L, W.BF16, 2)
    hd, H, Hkv = geo[1], geo[2], geo[3]
    rng = np.random.default_rng(0)
    raw = [W.normal((B, T, h, hd), 3 + i, W.BF16).to(DEV) for i, h in enumerate((H, Hkv, Hkv))]
    qw, kw = W.norm_weight(hd, 7).to(DEV), W.norm_weight(hd, 8).to(DEV)
    d, s = (i32(x) for x in ids(rng, B, L, 40, 20))
    start, lens, begin, end = i32([0, 0]), i32([T, T - 9]), i32(np.zeros((B, T))), i32(np.zeros((B, T)))
    pos, rows = i32(np.arange(T)[None].repeat(B, 0)[None].repeat(3, 0)), i32(np.arange(T)[None].repeat(B, 0))
    axes = G.rope_axes(3, axes_of(c.g, 3, True), hd)
    mods = G.score_mods(50.0, None, begin, end)
    q_out, out = torch.empty_like(raw[0]), torch.empty_like(raw[0])
    dec = torch.empty((B, H, hd), dtype=torch.bfloat16, device=DEV)
    wide = params_of(geometry(W.SLIDING, hd, H=H, Hkv=Hkv, window=4000, dtype=W.BF16))   # (its decode needs a workspace)
    size = G.g4_attn_decode_mods_workspace_size(wide, B, L)
    assert size > 0
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)

    def run():
        G.g4_attn_visible_ranges(geo[4], start, lens, d, s, L, B, T, begin, end)
        G.g4_kv_append_normrope_axes(c.params, c.table, 0, axes, *raw, qw, kw, pos, rows, B, T, q_out)
        G.g4_attn_prefill_mods(c.params, c.table, 0, mods, q_out, start, B, T, out)
        G.g4_attn_decode_mods(wide, c.table, 0, G.score_mods(20.0), q_out[:, 5].contiguous(), lens, B, L, dec, ws, size)

    run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run()
    torch.cuda.synchronize()
    for turn in range(3):
        for i, x in enumerate(raw):
            x.copy_(W.normal(tuple(x.shape), 100 * turn + i, W.BF16))
        lens.copy_(i32([T - turn, 20 + turn]))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (begin, end, q_out, out, dec, c.dk[:, :, :T], c.dv[:, :, :T])]
        run()
        torch.cuda.synchronize()
        for a, b in zip(got, (begin, end, q_out, out, dec, c.dk[:, :, :T], c.dv[:, :, :T])):
            assert torch.equal(a, b)


def test_one_workspace_for_all_decodes_in_turn():
    """Calls of other layers, batches and lengths in turn leave a workspace ready for the next."""
    cases = [(GEOS[1], [3000, 17]), ((W.FULL, 64, 8, 8, 0), [900] * 40), (GEOS[2], [5000]), (GEOS[4], [600, 1, 2000])]
    runs = []
    for i, (geo, lens) in enumerate(cases):
        c = Case(geo, lens, max(lens), W.BF16, 20 + i)
        q = unit((len(lens), geo[2], geo[1]), 40 + i, W.BF16).to(DEV)
        runs.append((c, q, lens, G.g4_attn_decode_mods_workspace_size(c.params, len(lens), max(lens))))
    size = max(r[3] for r in runs)
    shared = torch.zeros(size, dtype=torch.uint8, device=DEV)
    for c, q, lens, need in runs * 2:
        outs = []
        for ws in (torch.zeros(max(16, need), dtype=torch.uint8, device=DEV), shared):
            out = torch.empty_like(q)
            G.g4_attn_decode_mods(c.params, c.table, 0, G.score_mods(30.0), q, i32(lens), len(lens), max(lens), out, ws,
                                  ws.numel())
            outs.append(out)
        assert torch.equal(*outs)


def test_lengths_set_by_the_kernel_before():
    """Lengths and first keys that the work right before the call writes."""
    geo = GEOS[1]
    c = Case(geo, [900, 900, 900], 900, W.BF16, 3)
    q = unit((3, geo[2], geo[1]), 5, W.BF16).to(DEV)
    size = G.g4_attn_decode_mods_workspace_size(c.params, 3, 900)
    ws = torch.zeros(max(16, size), dtype=torch.uint8, device=DEV)
    lens, begin = i32([1, 1, 1]), i32([0, 0, 0])
    rng = np.random.default_rng(1)
    for _ in range(20):
        n = rng.integers(0, 901, 3)
        b = (n * rng.random(3)).astype(int)
        want = torch.empty_like(q)
        fresh = i32(n), i32(b)
        torch.cuda.synchronize()
        mods = G.score_mods(0.0, None, fresh[1])
        G.g4_attn_decode_mods(c.params, c.table, 0, mods, q, fresh[0], 3, 900, want, ws, size)
        out = torch.empty_like(q)
        lens.copy_(fresh[0])
        begin.copy_(fresh[1])
        G.g4_attn_decode_mods(c.params, c.table, 0, G.score_mods(0.0, None, begin), q, lens, 3, 900, out, ws, size)
        assert torch.equal(out, want)


def test_no_mods_are_the_plain_calls_within_their_rounding():
    """mods=None: the plain calls' outputs, which differ by roundings only."""
    geo = GEOS[4]
    c = Case(geo, [300, 200], 300, W.BF16, 4)
    q = unit((2, 100, geo[2], geo[1]), 5, W.BF16)
    out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    G.g4_attn_prefill_mods(c.params, c.table, 0, None, q.to(DEV), i32([200, 100]), 2, 100, out)
    at = np.array([[200], [100]]) + np.arange(100)[None]
    lo, hi = M.default_intervals(at, geo[0], geo[4])
    want, mass, size = c.reference(f64(q), at, lo, hi, [300, 200], 0.0, None)
    check(f64(out), want, mass, size, c.g, 300, 0.0, True, "none")
    d = torch.empty((2, geo[2], geo[1]), dtype=q.dtype, device=DEV)
    n = G.g4_attn_decode_mods_workspace_size(c.params, 2, 300)
    ws = torch.zeros(max(16, n), dtype=torch.uint8, device=DEV)
    G.g4_attn_decode_mods(c.params, c.table, 0, None, q[:, -1].contiguous().to(DEV), i32([300, 200]), 2, 300, d, ws, n)
    want, mass, size = c.reference(f64(q)[:, -1:], at[:, -1:], lo[:, -1:], hi[:, -1:], [300, 200], 0.0, None)
    check(f64(d)[:, None], want, mass, size, c.g, 300, 0.0, False, "none")


def test_intervals_straight_into_the_attention():
    """Each call right behind the one that writes its intervals, with the documents changed in between: as with a
    synchronisation."""
    geo, B, T, L = GEOS[1], 3, 40, 900
    c = Case(geo, [L] * B, L, W.BF16, 3)
    rng = np.random.default_rng(2)
    q = unit((B, T, geo[2], geo[1]), 5, W.BF16).to(DEV)
    size = G.g4_attn_decode_mods_workspace_size(c.params, B, L)
    ws = torch.zeros(max(16, size), dtype=torch.uint8, device=DEV)
    doc, lens, start = i32(np.zeros((B, L))), i32([0] * B), i32([0] * B)
    begin, end, last = i32(np.zeros((B, T))), i32(np.zeros((B, T))), i32([0] * B)
    one, one_end = i32(np.zeros((B, 1))), i32(np.zeros((B, 1)))
    for _ in range(12):
        n = rng.integers(T, L + 1, B)
        doc.copy_(i32(np.cumsum(rng.random((B, L)) < 0.01, 1)))
        lens.copy_(i32(n))
        start.copy_(i32(n - T))
        last.copy_(i32(n - 1))
        outs = []
        for wait in (False, True):
            outs.append([torch.empty_like(q), torch.empty_like(q[:, 0])])
            begin.zero_(), end.zero_(), one.zero_()
            torch.cuda.synchronize()
            G.g4_attn_visible_ranges(0, start, lens, doc, None, L, B, T, begin, end)
            if wait:
                torch.cuda.synchronize()
            G.g4_attn_prefill_mods(c.params, c.table, 0, G.score_mods(0.0, None, begin, end), q, start, B, T, outs[-1][0])
            G.g4_attn_visible_ranges(0, last, lens, doc, None, L, B, 1, one, one_end)
            if wait:
                torch.cuda.synchronize()
            G.g4_attn_decode_mods(c.params, c.table, 0, G.score_mods(0.0, None, one.view(B)), q[:, -1].contiguous(), lens, B,
                                  L, outs[-1][1], ws, size)
            torch.cuda.synchronize()
        for a, b in zip(*outs):
            assert torch.equal(a, b) and torch.isfinite(a).all()


def test_two_streams_at_once():
    """Prefills and decodes (a workspace each) on two streams at a time give what they give alone."""
    geo, T, L = GEOS[4], 700, 900
    c = Case(geo, [L, L], L, W.BF16, 3)
    size = G.g4_attn_decode_mods_workspace_size(c.params, 2, L)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    qs = [unit((2, T, geo[2], geo[1]), 5 + i, W.BF16).to(DEV) for i in range(2)]
    last = [q[:, -1].contiguous() for q in qs]
    starts, lens = [i32([200, 100]), i32([0, 150])], [i32([900, 800]), i32([300, 5])]
    mods = [G.score_mods(30.0), G.score_mods(0.0, torch.tensor(SLOPES(geo[2]), dtype=torch.float32, device=DEV))]
    spaces = [torch.zeros(max(16, size), dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [[(torch.empty_like(q), torch.empty_like(x)) for q, x in zip(qs, last)] for _ in range(5)]
    torch.cuda.synchronize()
    for turn, pair in enumerate(outs):
        for i, (o, d) in enumerate(pair):
            G.g4_attn_prefill_mods(c.params, c.table, 0, mods[i], qs[i], starts[i], 2, T, o, stream=streams[i])
            G.g4_attn_decode_mods(c.params, c.table, 0, mods[i], last[i], lens[i], 2, L, d, spaces[i], size, stream=streams[i])
            if turn == 0:
                torch.cuda.synchronize()
    torch.cuda.synchronize()
    for pair in outs[1:]:
        for (o, d), (o0, d0) in zip(pair, outs[0]):
            assert torch.equal(o, o0) and torch.equal(d, d0)


@pytest.mark.parametrize("geo", [GEOS[1], GEOS[2], GEOS[3], (W.FULL, 256, 3, 3, 0)])
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("B,most", [(70, 5), (70, 64), (70, 65), (610, 5), (610, 40)])
def test_decode_of_many_short_sequences(geo, dtype, B, most):
    """A CTA for every unit, or more units than CTAs; sequences of no, one and up to `most` keys."""
    lens = [i % (most + 1) for i in range(B)]
    c = Case(geo, [max(1, n) for n in lens], most, dtype, 12)
    q = unit((B, geo[2], geo[1]), 3, dtype)
    size = G.g4_attn_decode_mods_workspace_size(c.params, B, most)
    ws = torch.zeros(max(16, size), dtype=torch.uint8, device=DEV)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    begin = [n // 3 for n in lens]
    G.g4_attn_decode_mods(c.params, c.table, 0, G.score_mods(9.0, None, i32(begin)), q.to(DEV), i32(lens), B, most, out, ws, size)
    at = np.asarray(lens)[:, None] - 1
    lo, hi = M.default_intervals(at, geo[0], geo[4])
    want, mass, mag = c.reference(f64(q)[:, None], at, np.maximum(lo, np.asarray(begin)[:, None]), hi, lens, 9.0, None)
    check(f64(out)[:, None], want, mass, mag, c.g, most, 9.0, False, geo)
