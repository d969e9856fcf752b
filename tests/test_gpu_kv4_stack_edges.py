"""PagedAttnStack off its usual steps, on the GPU: prompts of one token through prefill, captured prefills."""

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


def test_a_graph_keeps_its_prefill_workspace():
    """A captured prefill repeats its bits after longer ones, and writes to no memory that others hold by then."""
    B, H, Hkv, l, T = CFG["B"], CFG["H"], CFG["Hkv"], 1, 6
    st = S.PagedAttnStack(CFG, max_len=160, n_blocks=26, block_size=32, device=DEV)
    st.assign(i32([T] * B), T)
    q, k, v = (bf16_normal((B, T, n, 128), i).to(DEV) for i, n in enumerate((H, Hkv, Hkv)))
    w = W.norm_weight(128, 4).to(DEV)
    q_out, out = torch.empty_like(q), torch.empty_like(q)
    st.append(l, q, k, v, w, w, T, q_out)
    st.prefill_attn(l, q_out, T, out)
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.prefill_attn(l, q_out, T, out)
    size = st._prefill_ws.numel()
    at = st._prefill_ws.data_ptr()
    long = torch.zeros((B, 120, H, 128), dtype=torch.bfloat16, device=DEV)
    for n in (60, 120):
        st.prefill_attn(l, long[:, :n].contiguous(), n, long[:, :n].contiguous())
    assert st._prefill_ws.data_ptr() != at
    others = [torch.full((size,), 255, dtype=torch.uint8, device=DEV) for _ in range(8)]
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(bool((x == 255).all()) for x in others)
