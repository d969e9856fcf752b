"""PagedAttnStack off its usual steps, on the GPU: prompts of one token through prefill."""

import numpy as np
import pytest

from gemma_dual_geometry_gb300 import build as g4build
from gemma_dual_geometry_gb300 import stack as S

from kv4_common import DEV, G, K, O, W, bf16_normal, f64, i32, torch
from test_gpu_kv4_stack import CFG

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    g4build.build()
    G.lib()
    yield
    assert G.g4_take_device_error() == 0


def test_prompts_of_one_token():
    """Attention over one key is its value, whatever the query."""
    B, H, Hkv = CFG["B"], CFG["H"], CFG["Hkv"]
    st = S.PagedAttnStack(CFG, max_len=160, n_blocks=26, block_size=32, device=DEV)
    st.assign(i32([1] * B), 1)
    for l in (0, 1):
        g = st.geo[l]
        hd = g["head_dim"]
        q, k, v = (bf16_normal((B, 1, n, hd), 5 * l + i).to(DEV) for i, n in enumerate((H, Hkv, Hkv)))
        w = W.norm_weight(hd, l).to(DEV)
        q_out, out = torch.empty_like(q), torch.empty_like(q)
        st.append(l, q, k, v, w, w, 1, q_out)
        st.prefill_attn(l, q_out, 1, out)
        _, vn = O.normrope_kv(f64(k), f64(v), f64(w), np.zeros((B, 1), int), hd, g["theta"], g["rotary_fraction"], g["eps"])
        want = np.repeat(K.values(*K.quantise(O.round_bf16(vn))), H // Hkv, 2)
        assert np.array_equal(f64(out), want)   # (the weight of the one key is its own sum: the quotient is exact)
