"""Modified scores, intervals and several axes where offsets pass 32 bits: caches, queries and rows of more than 2^31
elements.  What lies at their far end is compared with the same rows in small buffers (distances, not positions, count)."""

import numpy as np
import pytest

from gemma_dual_geometry_gb300 import build as g4build
from gpu_common import DEV, G, W, geometry, params_of, torch
from test_gpu_mods import SLOPES, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    g4build.build()
    G.lib()
    yield
    assert G.g4_take_device_error() == 0
    torch.cuda.empty_cache()


def slopes(H):
    return torch.tensor(SLOPES(H), dtype=torch.float32, device=DEV)


def cache(B, Hkv, L, hd, dtype, layer_type=W.FULL):
    k, v = (torch.zeros((B, Hkv, L, hd), dtype=dtype, device=DEV) for _ in range(2))
    tab = G.cache_table(1)
    G.set_cache(tab, 0, k, v, layer_type, hd, Hkv, L, B, W.BF16 if dtype == torch.bfloat16 else W.F32)
    return k, v, tab


@pytest.mark.parametrize("hd,dtype", [(512, torch.bfloat16), (128, torch.float32)])
def test_keys_at_the_end_of_a_long_cache(hd, dtype):
    """Decode, prefill and append at positions whose elements lie past 2^31 of the cache, against a cache of 700 rows."""
    H, Hkv, n, T = 8, 2, 700, 40
    L = (1 << 31) // (Hkv * hd) + 1000    # (the second kv head's rows lie past 2^30 elements, its last ones past 2^31)
    at = L - n
    g = geometry(W.FULL, hd, H=H, Hkv=Hkv, dtype=W.BF16 if dtype == torch.bfloat16 else W.F32)
    p = params_of(g)
    torch.manual_seed(1)
    rows = [torch.randn((1, Hkv, n, hd), device=DEV).to(dtype) for _ in range(2)]
    q = (torch.randn((1, T, H, hd), device=DEV) / hd ** 0.5).to(dtype)
    raw = [torch.randn((1, T, h, hd), device=DEV).to(dtype) for h in (H, Hkv, Hkv)]
    w = torch.ones(hd, device=DEV)
    outs = []
    for first, length in ((at, L), (0, n)):
        k, v, tab = cache(1, Hkv, length, hd, dtype)
        k[:, :, first:], v[:, :, first:] = rows
        axes = G.rope_axes(2, [j % 2 for j in range(hd // 2)], hd)
        pos = i32(np.arange(2 * T).reshape(2, 1, T))
        q_out = torch.empty_like(raw[0])
        G.g4_kv_append_normrope_axes(p, tab, 0, axes, *raw, w, w, pos, i32(first + n - T + np.arange(T)[None]), 1, T, q_out)
        begin = i32(first + np.arange(T)[None])
        pre, dec = torch.empty_like(q), torch.empty((1, H, hd), dtype=dtype, device=DEV)
        G.g4_attn_prefill_mods(p, tab, 0, G.score_mods(20.0, slopes(H), begin), q, i32([first + n - T]), 1, T, pre)
        size = G.g4_attn_decode_mods_workspace_size(p, 1, length)
        ws = torch.zeros(max(16, size), dtype=torch.uint8, device=DEV)
        G.g4_attn_decode_mods(p, tab, 0, G.score_mods(20.0, slopes(H), i32([first + 3])), q[:, 0].contiguous(), i32([length]), 1,
                              length, dec, ws, size)
        outs.append((k[:, :, first:].clone(), v[:, :, first:].clone(), q_out, pre, dec))
        if first:
            assert not k[:, :, :first].any() and not v[:, :, :first].any()
        del k, v, tab
        torch.cuda.empty_cache()
    for a, b in zip(outs[0][:3], outs[1][:3]):
        assert torch.equal(a, b)
    # (other tiles and splits: prefill's weights, rounded to bf16 from another base, are each off by 2^-8 on either side of a
    # mean of |v| < 5, 2 x 2^-8 x 5 in all; float32 sums of 700 terms in another order by 700 x 2^-24 x 5 x 2 at most)
    for a, b in zip(outs[0][3:], outs[1][3:]):
        assert torch.isfinite(a).all() and (a.float() - b.float()).abs().max() < (2.0 ** -7 * 5 + 2.0 ** -8 if dtype == torch.bfloat16 else 5e-4)


def test_many_queries():
    """Queries and outputs of more than 2^31 elements: the last sequence's, against a call of its own."""
    H, Hkv, hd, T, B = 16, 8, 512, 66000, 4
    g = geometry(W.SLIDING, hd, H=H, Hkv=Hkv, window=60, dtype=W.BF16)
    p = params_of(g)
    torch.manual_seed(2)
    k, v, tab = cache(B, Hkv, T, hd, torch.bfloat16, W.SLIDING)
    k.normal_(), v.normal_()
    q = torch.empty((B, T, H, hd), dtype=torch.bfloat16, device=DEV).normal_(std=0.05)
    assert q.numel() > 2 ** 31 and k.numel() > 2 ** 30
    out = torch.empty_like(q)
    G.g4_attn_prefill_mods(p, tab, 0, G.score_mods(30.0), q, i32([0] * B), B, T, out)
    one = G.cache_table(1)
    G.set_cache(one, 0, k[-1:], v[-1:], W.SLIDING, hd, Hkv, T, 1, W.BF16)
    last = torch.empty_like(q[-1:])
    G.g4_attn_prefill_mods(p, one, 0, G.score_mods(30.0), q[-1:], i32([0]), 1, T, last)
    assert torch.equal(out[-1:], last)
    # and the append of as many rows, in place and apart
    w = torch.ones(hd, device=DEV)
    pos = i32(np.arange(T)[None].repeat(B, 0))
    axes = G.rope_axes(1, [0] * (hd // 2), hd)
    shared = G.layer_params(W.SLIDING, hd, H, Hkv, 60, g["theta"], 1.0, W.EPS, 1.0, 0, W.BF16)
    tab2 = G.cache_table(2)
    G.set_cache(tab2, 0, k, v, W.SLIDING, hd, Hkv, T, B, W.BF16)
    G.g4_kv_append_normrope_axes(shared, tab2, 1, axes, q, None, None, w, None, i32(pos.cpu().numpy()[None]), None, B, T, out)
    G.g4_kv_append_normrope(shared, tab2, 1, q, None, None, w, None, pos, B, T, q)
    assert torch.equal(out, q)


def test_the_longest_rows_of_ids():
    """Rows of 2^24 positions: whole documents and spans across all of a cluster's tiles."""
    L, T = 1 << 24, 5000
    doc = torch.zeros((2, L), dtype=torch.int32, device=DEV)
    span = torch.full((2, L), -1, dtype=torch.int32, device=DEV)
    doc[1, 12345678:] = 1
    span[0, 777:L - 100] = 4
    for start, window in (([0, L - T], 0), ([L - T, 12345678 - 10], 512), ([L // 2, 0], 100)):
        begin, end = (torch.empty((2, T), dtype=torch.int32, device=DEV) for _ in range(2))
        G.g4_attn_visible_ranges(window, i32(start), i32([L, L - 5]), doc, span, L, 2, T, begin, end)
        at = np.asarray(start)[:, None] + np.arange(T)[None]
        lo = np.where(at < 12345678, 0, 12345678) * np.array([[0], [1]])
        hi = at + 1
        if window:
            lo = np.maximum(lo, at - window + 1)
        inside = (at[0] >= 777) & (at[0] < L - 100)
        lo[0], hi[0] = np.where(inside, np.minimum(lo[0], 777), lo[0]), np.where(inside, L - 100, hi[0])
        gone = at[1] >= L - 5
        lo[1], hi[1] = np.where(gone, 0, lo[1]), np.where(gone, 0, hi[1])
        assert np.array_equal(begin.cpu().numpy(), lo) and np.array_equal(end.cpu().numpy(), hi)
