"""g4_kv_append_normrope with q_out = q_in, as the header allows it: the same bits as with a buffer of its own.  (Values
that float32 leaves open are formed from the inputs again after the row's others have been stored.)"""

import numpy as np
import pytest

from gemma_dual_geometry_gb300 import build as g4build
from gpu_common import DEV, G, O, W, f64, geometry, params_of, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    g4build.build()
    G.lib()
    yield
    assert G.g4_take_device_error() == 0


@pytest.mark.parametrize("geo", [(W.SLIDING, 256, 8, 2), (W.FULL, 512, 8, 2), (W.FULL, 128, 8, 1), (W.SLIDING, 64, 3, 3)])
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("B,T", [(9, 1), (3, 150), (1, 1200)])
@pytest.mark.parametrize("shared", [False, True])
def test_append_in_place(geo, dtype, B, T, shared):
    g = geometry(geo[0], geo[1], H=geo[2], Hkv=geo[3], window=T, dtype=dtype)
    hd, H, Hkv = g["head_dim"], g["n_heads"], g["n_kv_heads"]
    x = [W.normal((B, T, h, hd), 3 + h, dtype).to(DEV) for h in (H, Hkv, Hkv)]
    qw, kw = W.norm_weight(hd, 7), W.norm_weight(hd, 8)
    pos = np.random.default_rng(T).integers(0, 10, B)[:, None] + np.arange(T)[None]
    d_pos = torch.tensor(pos, dtype=torch.int32, device=DEV)
    p = params_of(g, 0 if shared else -1)
    caches = []
    for _ in range(2):
        c = [torch.zeros((B, Hkv, T + 10, hd), dtype=x[0].dtype, device=DEV) for _ in range(2)]
        tab = G.cache_table(2)
        G.set_cache(tab, 0, *c, g["layer_type"], hd, Hkv, T + 10, B, dtype)
        caches.append((tab, c))
    kv = (None, None, qw.to(DEV), None) if shared else (x[1], x[2], qw.to(DEV), kw.to(DEV))
    apart, same = torch.empty_like(x[0]), x[0].clone()
    layer = 1 if shared else 0
    G.g4_kv_append_normrope(p, caches[0][0], layer, x[0], *kv, d_pos, B, T, apart)
    G.g4_kv_append_normrope(p, caches[1][0], layer, same, *kv, d_pos, B, T, same)
    assert torch.equal(apart, same)
    assert all(torch.equal(a, b) for a, b in zip(caches[0][1], caches[1][1]))
    if dtype == W.BF16:
        want = O.normrope_q(f64(x[0]), f64(qw), pos, hd, g["theta"], g["rotary_fraction"], g["eps"])
        assert np.array_equal(f64(same), O.round_bf16(want))
