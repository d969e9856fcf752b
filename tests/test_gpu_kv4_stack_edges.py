"""PagedAttnStack off its usual steps, on the GPU: prompts of one token through prefill, captured prefills,
streams of its own."""

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


def rows(T, hd, seed):
    return [bf16_normal((CFG["B"], T, n, hd), seed + i).to(DEV) for i, n in enumerate((CFG["H"], CFG["Hkv"], CFG["Hkv"]))]


def run(st, l, data, w, stream):
    """A prompt of 40 tokens per sequence, then a step: what the step's attention gives."""
    B, H, hd = CFG["B"], CFG["H"], st.geo[l]["head_dim"]
    q_out, out = (torch.empty((B, 1, H, hd), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for T, want, (q, k, v) in ((40, i32([40] * B), data[0]), (1, i32([41] * B), data[1])):
        qo = torch.empty_like(q)
        if stream is not None:
            stream.wait_stream(torch.cuda.default_stream())   # what the caller made; not what the stack did
        st.assign(want, T, stream=stream)
        st.append(l, q, k, v, w, w, T, qo if T > 1 else q_out, stream=stream)
        for t in (want, qo):
            if stream is not None:
                t.record_stream(stream)
    st.decode_attn(l, q_out, out, stream=stream)
    if stream is not None:
        q_out.record_stream(stream)
    return out


def test_first_calls_on_a_stream_of_its_own():
    """The constructor's stream is still busy when the first call goes to another one: the free list, the lengths
    and the counters of decode's workspace are in place all the same.  (The caller does not wait for the
    constructor's stream here; its tensors were made before.)"""
    l = 1
    data, w = [rows(40, 128, 1), rows(1, 128, 5)], W.norm_weight(128, 4).to(DEV)
    want = run(S.PagedAttnStack(CFG, max_len=160, n_blocks=26, block_size=32, device=DEV), l, data, w, None)
    lens = [i32([40] * CFG["B"]), i32([41] * CFG["B"])]
    q_out, out, qo = torch.empty_like(want), torch.empty_like(want), torch.empty_like(data[0][0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)   # about 20 ms, on the constructor's stream
    st = S.PagedAttnStack(CFG, max_len=160, n_blocks=26, block_size=32, device=DEV)
    for n, T in zip(lens, (40, 1)):
        q, k, v = data[T == 1]
        st.assign(n, T, stream=side)
        st.append(l, q, k, v, w, w, T, qo if T > 1 else q_out, stream=side)
    st.decode_attn(l, q_out, out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    st.decode_attn(l, q_out, out.zero_())   # (the counters are as a call leaves them)
    assert torch.equal(out, want)


def test_a_stack_that_goes_before_its_work_is_done():
    """Its memory is not handed out while a stream that it was used on is still at work."""
    l = 1
    data, w = [rows(40, 128, 1), rows(1, 128, 5)], W.norm_weight(128, 4).to(DEV)
    want = run(S.PagedAttnStack(CFG, max_len=160, n_blocks=26, block_size=32, device=DEV), l, data, w, None)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    st = S.PagedAttnStack(CFG, max_len=160, n_blocks=26, block_size=32, device=DEV)
    sizes = [t.numel() * t.element_size() for t in st._buffers()]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    out = run(st, l, data, w, side)
    out.record_stream(side)
    del st
    others = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(bool((x == 255).all()) for x in others)


def test_a_workspace_outgrown_while_a_stream_known_by_address_uses_it():
    """A longer prefill on the current stream replaces the workspace that a side stream, given by its address, is
    still to write: what is taken after that is not written to."""
    l, T = 1, 30
    data, w = rows(T, 128, 1), W.norm_weight(128, 4).to(DEV)
    st = S.PagedAttnStack(CFG, max_len=160, n_blocks=26, block_size=32, device=DEV)
    st.assign(i32([T] * CFG["B"]), T)
    q_out, out, late = (torch.empty_like(data[0]) for _ in range(3))
    st.append(l, *data, w, w, T, q_out)
    st.prefill_attn(l, q_out, T, out)
    size = st._prefill_ws.numel()
    long = torch.zeros((CFG["B"], 120, CFG["H"], 128), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    st.prefill_attn(l, q_out, T, late, stream=side.cuda_stream)
    st.prefill_attn(l, long, 120, long)
    others = [torch.full((size,), 255, dtype=torch.uint8, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(late, out)
    assert all(bool((x == 255).all()) for x in others)
