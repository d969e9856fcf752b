"""Prefill with modified scores over rings: positions up to the last one that 32 bits hold, and intervals of the caller's own."""

import numpy as np
import pytest

from gemma_dual_geometry_gb300 import build as g4build
from gpu_common import DEV, G, O, W, f64, torch
from oracle import mods_oracle as M
from test_gpu_mods import GEOS, SLOPES, Case, check, i32, unit

pytestmark = pytest.mark.gpu
LAST = 2 ** 31 - 1   # (no position: one past the last)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    g4build.build()
    G.lib()
    yield
    assert G.g4_take_device_error() == 0


def run(c, start, T, cap=0.0, bias=False, begin=None, end=None, seed=3, rows=None):
    """Prefill of T tokens from `start` on a ring Case against the oracle; `rows`: which of the tokens are compared."""
    start, g = np.asarray(start, np.int64), c.g
    B, at = len(start), start[:, None] + np.arange(T)[None]
    q = unit((B, T, g["n_heads"], g["head_dim"]), seed, c.dtype)
    slopes = SLOPES(g["n_heads"]) if bias else None
    mods = G.score_mods(cap, None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device=DEV),
                        None if begin is None else i32(begin), None if end is None else i32(end))
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=DEV)
    G.g4_attn_prefill_mods(c.params, c.table, 0, mods, q.to(DEV), i32(start), B, T, out)
    lo, hi = M.default_intervals(at, g["layer_type"], g["window"])
    lo, hi = lo if begin is None else np.asarray(begin), hi if end is None else np.asarray(end)
    some = np.arange(T) if rows is None else rows
    want, mass, size = c.reference(f64(q)[:, some], at[:, some], lo[:, some], hi[:, some], start + T, cap, slopes)
    check(f64(out)[:, some], want, mass, size, g, c.Lmax, cap, c.dtype == W.BF16, (start, T, cap, bias))
    return f64(out), lo, hi


def ring(geo, B, rows, dtype, seed=2):
    return Case(geo, [rows] * B, rows, dtype, seed, ring=True)


# a chunk's tokens, its ring's rows: one tile, two, and three, the last tile full or not
NEAR = [((W.SLIDING, 256, 4, 2, 40), 80, 256), ((W.SLIDING, 64, 2, 2, 17), 1, 128), ((W.SLIDING, 64, 3, 3, 33), 130, 256),
        ((W.SLIDING, 512, 2, 1, 100), 100, 384), ((W.SLIDING, 128, 4, 4, 300), 300, 640)]


@pytest.mark.parametrize("geo,T,rows", NEAR)
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, True)])
def test_chunks_at_the_last_positions(geo, T, rows, dtype, cap, bias):
    """Chunks whose last position is 2^31 - 2, or that end at or beside the last whole tile."""
    starts = [LAST - T, LAST - T - 1, LAST - T - 127, LAST - T - 128, LAST - T - 129]
    c = ring(geo, len(starts), rows, dtype)
    run(c, starts, T, cap, bias)
    # and with intervals given: to the end of what is held, from what the ring still has
    at = np.asarray(starts)[:, None] + np.arange(T)[None]
    begin = np.maximum(at - rows - 5, 0) + np.arange(T)[None] % 90
    run(c, starts, T, cap, bias, begin, np.minimum(at + 1 + np.arange(T)[None] % 50, LAST))


@pytest.mark.parametrize("geo,T,rows", NEAR)
def test_plain_chunks_at_the_last_positions(geo, T, rows):
    """g4_attn_prefill, whose items are found the same way."""
    starts = np.array([LAST - T, LAST - T - 1, LAST - T - 127, LAST - T - 128], np.int64)
    c = ring(geo, len(starts), rows, W.BF16)
    q = unit((len(starts), T, geo[2], geo[1]), 3, W.BF16)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=DEV)
    G.g4_attn_prefill(c.params, c.table, 0, q.to(DEV), i32(starts), len(starts), T, out)
    at = starts[:, None] + np.arange(T)[None]
    lo, hi = M.default_intervals(at, geo[0], geo[4])
    want, mass, size = c.reference(f64(q), at, lo, hi, starts + T, 0.0, None)
    check(f64(out), want, mass, size, c.g, rows, 0.0, True, (geo, T))


@pytest.mark.parametrize("geo,T,rows", [n for n in NEAR if n[1] > 1])
@pytest.mark.parametrize("start", ["last", 3000])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, True)])
def test_rows_formed_again_on_a_ring(geo, T, rows, start, cap, bias):
    """NaN and an infinity in the last keys' values, which some of a tile's queries see: the others' rows are right, up to
    the last position (keys are counted in eights there), and where the ring wraps."""
    start = LAST - T if start == "last" else start
    c = ring(geo, 1, rows, W.BF16)
    held = start + T
    c.dv[0, :, (held - 1) % rows] = float("nan")
    c.dv[0, :, (held - 20) % rows] = float("inf")
    at = start + np.arange(T)
    seen = np.where(np.arange(T) % 3 == 0, held, held - 1 - np.arange(T) % 3)[None]
    seen = np.where((np.arange(T) % 5 == 0)[None], held - 20 - np.arange(T)[None] % 40, seen)
    begin = np.where(np.arange(T) % 4 == 1, held - 19, held - np.minimum(rows, 60 + np.arange(T)))[None]
    clean = ~((seen[0] == held) | ((begin[0] <= held - 20) & (seen[0] > held - 20)))
    assert 0.2 < clean.mean() < 0.8
    out, _, _ = run(c, [start], T, cap, bias, begin, seen, rows=np.flatnonzero(clean))
    assert not np.isfinite(out[0, ~clean]).any()
    # the causal form: the last token alone sees the last key
    c.dv[0, :, (held - 20) % rows] = 1.0
    c.v.copy_(c.dv)
    out, _, _ = run(c, [start], T, cap, bias, rows=np.arange(T - 1))
    assert np.isnan(out[0, T - 1]).all()


@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("geo,T,rows", [((W.SLIDING, 256, 4, 2, 200), 250, 256), ((W.SLIDING, 64, 8, 1, 100), 384, 384),
                                        ((W.SLIDING, 512, 2, 2, 33), 129, 384), ((W.SLIDING, 128, 3, 3, 128), 1, 128)])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (50.0, True)])
def test_intervals_of_the_callers_own(geo, T, rows, dtype, cap, bias):
    """Intervals that begin before what the ring still holds, that end past the query or past the last position, that are
    empty; chunks that leave no room for the layer's window; rings that are not full, and that wrap inside a tile."""
    starts = np.array([0, 3, 1000, 777, 2 * rows, 12345])
    B, at = len(starts), starts[:, None] + np.arange(T)[None]
    rng = np.random.default_rng(T + rows)
    begin = at - rng.integers(0, 2 * rows, at.shape)
    end = at + rng.integers(-rows // 2, rows, at.shape)
    begin[:, T // 3], end[:, T // 3] = -2 ** 31, 2 ** 31 - 1      # all that is held
    end[:, T // 2:T // 2 + 3] = (starts + T - rows)[:, None]      # nothing that is
    out, lo, hi = run(ring(geo, B, rows, dtype), starts, T, cap, bias, begin, end)
    held = (starts + T)[:, None]
    empty = np.minimum(hi, held) <= np.maximum(lo, np.maximum(held - rows, 0))
    assert empty.any() and (out[empty] == 0).all()
    run(ring(geo, B, rows, dtype), starts, T, cap, bias, begin, None)
