"""Keys that a query sees whose scores are minus infinity: they weigh nothing, wherever they lie among its keys.  The
steepest slopes, next to infinity."""

import numpy as np
import pytest

from gemma_dual_geometry_gb300 import build as g4build
from gpu_common import DEV, G, W, f64, torch
from test_gpu_mods import GEOS, SLOPES, Case, check, i32, unit

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    g4build.build()
    G.lib()
    yield
    assert G.g4_take_device_error() == 0


def case(geo, n, low, dtype):
    """A sequence of n keys whose first `low` score minus infinity with every query below."""
    c = Case(geo, [n], n, dtype, 8)
    c.dk[0, :, :low, 5] = float("-inf")
    return c


def queries(geo, T, dtype):
    q = unit((1, T, geo[2], geo[1]), 3, dtype)
    q[..., 5] = q[..., 5].abs() + 0.25
    return q


def mods_of(geo, bias, *given):
    slopes = SLOPES(geo[2]) if bias else None
    return slopes, G.score_mods(0.0, None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device=DEV), *given)


# (windows wide enough for the keys below)
WIDE = [(g[0], g[1], g[2], g[3], 4000 if g[0] == W.SLIDING else 0) for g in GEOS]


@pytest.mark.parametrize("geo", WIDE)
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("n,low", [(2, 1), (3, 1), (100, 99), (300, 1), (300, 40), (300, 200), (900, 833)])
@pytest.mark.parametrize("bias", [False, True])
def test_decode(geo, dtype, n, low, bias):
    c, q = case(geo, n, low, dtype), queries(geo, 1, dtype)
    slopes, mods = mods_of(geo, bias)
    size = G.g4_attn_decode_mods_workspace_size(c.params, 1, n)
    ws = torch.zeros(max(16, size), dtype=torch.uint8, device=DEV)
    out = torch.empty((1, geo[2], geo[1]), dtype=q.dtype, device=DEV)
    G.g4_attn_decode_mods(c.params, c.table, 0, mods, q[:, 0].contiguous().to(DEV), i32([n]), 1, n, out, ws, size)
    want, mass, mag = c.reference(f64(q), np.array([[n - 1]]), [[low]], [[n]], [n], 0.0, slopes)
    check(f64(out)[:, None], want, mass, mag, c.g, n, 0.0, False, (geo, n, low))


@pytest.mark.parametrize("geo", WIDE)
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("n,T,low", [(40, 5, 1), (300, 150, 149), (400, 150, 200)])
@pytest.mark.parametrize("bias", [False, True])
def test_prefill(geo, dtype, n, T, low, bias):
    """Causal rows, and rows that see the last keys too."""
    c, q = case(geo, n, low, dtype), queries(geo, T, dtype)
    at = n - T + np.arange(T)[None]
    for end in (at + 1, np.full((1, T), n)):
        slopes, mods = mods_of(geo, bias, None, i32(end))
        out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
        G.g4_attn_prefill_mods(c.params, c.table, 0, mods, q.to(DEV), i32([n - T]), 1, T, out)
        want, mass, size = c.reference(f64(q), at, np.full((1, T), low), end, [n], 0.0, slopes)
        check(f64(out), want, mass, size, c.g, n, 0.0, dtype == W.BF16, (geo, n, low))


@pytest.mark.parametrize("geo", WIDE)
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
def test_nothing_but_such_keys(geo, dtype):
    """Rows of which every key scores minus infinity are zero, as those that see none."""
    n, T = 90, 4
    c, q = case(geo, n, n, dtype), queries(geo, T, dtype).to(DEV)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=DEV)
    G.g4_attn_prefill_mods(c.params, c.table, 0, None, q, i32([n - T]), 1, T, out)
    assert (out == 0).all()
    size = G.g4_attn_decode_mods_workspace_size(c.params, 1, n)
    ws = torch.zeros(max(16, size), dtype=torch.uint8, device=DEV)
    one = torch.full((1, geo[2], geo[1]), float("nan"), dtype=q.dtype, device=DEV)
    G.g4_attn_decode_mods(c.params, c.table, 0, None, q[:, 0].contiguous(), i32([n]), 1, n, one, ws, size)
    assert (one == 0).all()


@pytest.mark.parametrize("geo", WIDE)
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("n,T", [(2, 1), (130, 130), (400, 150), (900, 40)])
def test_the_steepest_slopes(geo, dtype, n, T):
    """Slopes of 2^64 leave the query's own key, of -2^64 the farthest one that it sees, to the bit."""
    c = Case(geo, [n], n, dtype, 8)
    q = unit((1, T, geo[2], geo[1]), 3, dtype).to(DEV)
    slopes = torch.tensor([2.0 ** 64 * (-1) ** h for h in range(geo[2])], device=DEV)
    at = torch.arange(n - T, n, device=DEV)
    group = geo[2] // geo[3]

    def rows(p, h):
        return c.dv[0, h // group, p]

    out = torch.empty_like(q)
    first = i32([[t % 7 for t in range(T)]]).clamp(max=n - T)
    G.g4_attn_prefill_mods(c.params, c.table, 0, G.score_mods(0.0, slopes, first), q, i32([n - T]), 1, T, out)
    for h in range(geo[2]):
        assert torch.equal(out[0, :, h], rows(at if h % 2 == 0 else first[0].long(), h))
    size = G.g4_attn_decode_mods_workspace_size(c.params, 1, n)
    ws = torch.zeros(max(16, size), dtype=torch.uint8, device=DEV)
    one = torch.empty((1, geo[2], geo[1]), dtype=q.dtype, device=DEV)
    G.g4_attn_decode_mods(c.params, c.table, 0, G.score_mods(0.0, slopes), q[:, 0].contiguous(), i32([n]), 1, n, one, ws, size)
    for h in range(geo[2]):
        assert torch.equal(one[0, h], rows(n - 1 if h % 2 == 0 else 0, h))
