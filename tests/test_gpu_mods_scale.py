"""Modified scores under a softmax scale other than 1, which the cap, the bias and the plain form each carry their own way."""

import numpy as np
import pytest

import gpu_common
import test_gpu_mods as T
from gemma_dual_geometry_gb300 import build as g4build
from gpu_common import DEV, G, W, f64, torch
from oracle import mods_oracle as M

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    g4build.build()
    G.lib()
    yield
    assert G.g4_take_device_error() == 0


class Scaled(T.Case):
    """A Case whose layer has the softmax scale `scale`."""

    def __init__(self, geo, lens, Lmax, dtype, seed, scale, ring=False):
        super().__init__(geo, lens, Lmax, dtype, seed, ring)
        self.scale = scale
        self.params = gpu_common.params_of(dict(self.g, attn_scale=scale))

    def reference(self, q, q_pos, begin, end, held, cap, slopes):
        B, n, H, hd = q.shape
        group = H // self.g["n_kv_heads"]
        out, mass, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3])
        k, v = f64(self.k), f64(self.v)
        for b in range(B):
            at = np.arange(int(held[b]))
            for h in range(H):
                out[b, :, h], mass[b, :, h], size[b, :, h] = M.attention_rows(
                    q[b, :, h], k[b, h // group, at], v[b, h // group, at], at, q_pos[b], begin[b], end[b], cap,
                    0.0 if slopes is None else slopes[h], self.scale)
        return out, mass, size


# scales of 1 / sqrt(head_dim) and of 1 / sqrt(a quarter of it), one above 1 (as with queries that carry their own factor), one
# that no power of two divides
@pytest.mark.parametrize("geo", T.GEOS)
@pytest.mark.parametrize("scale", [1.0, 2.0, "above", 0.3])
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (50.0, False), (0.0, True), (4.0, True)])
def test_scaled(geo, scale, dtype, cap, bias):
    scale = 1.75 if scale == "above" else 0.3 if scale == 0.3 else scale / np.sqrt(geo[1])
    scale = float(np.float32(scale))
    n, B, L = 150, 2, 300
    start = np.array([0, 130])
    lens = start + n
    c = Scaled(geo, lens, L, dtype, geo[1] + int(cap), scale)
    q = T.unit((B, n, geo[2], geo[1]), 9, dtype)
    at = start[:, None] + np.arange(n)[None]
    slopes = T.SLOPES(geo[2]) if bias else None
    d_slopes = None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device=DEV)
    lo, hi = M.default_intervals(at, geo[0], geo[4])
    for ends in (None, np.minimum(hi + np.arange(n)[None] % 3 * 20, lens[:, None])):
        out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
        mods = G.score_mods(cap, d_slopes, None, None if ends is None else T.i32(ends))
        G.g4_attn_prefill_mods(c.params, c.table, 0, mods, q.to(DEV), T.i32(start), B, n, out)
        want, mass, size = c.reference(f64(q), at, lo, hi if ends is None else ends, lens, cap, slopes)
        T.check(f64(out), want, mass, size, c.g, L, cap, dtype == W.BF16, ("prefill", geo, scale))
    # the last tokens as decodes
    size = G.g4_attn_decode_mods_workspace_size(c.params, B, L)
    ws = torch.zeros(max(16, size), dtype=torch.uint8, device=DEV)
    one = torch.empty((B, geo[2], geo[1]), dtype=q.dtype, device=DEV)
    G.g4_attn_decode_mods(c.params, c.table, 0, G.score_mods(cap, d_slopes), q[:, -1].contiguous().to(DEV), T.i32(lens), B, L,
                          one, ws, size)
    want, mass, mag = c.reference(f64(q)[:, -1:], at[:, -1:], lo[:, -1:], hi[:, -1:], lens, cap, slopes)
    T.check(f64(one)[:, None], want, mass, mag, c.g, L, cap, False, ("decode", geo, scale))
