"""One new token per sequence, as a decode and as a prefill of T = 1: the same keys, but where the header says otherwise."""

import numpy as np
import pytest

from gemma_dual_geometry_gb300 import build as g4build
from gpu_common import DEV, G, W, f64, torch
from oracle import mods_oracle as M
from test_gpu_mods import Case, check, i32, unit

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    g4build.build()
    G.lib()
    yield
    assert G.g4_take_device_error() == 0


# (the cluster kernel, the kernel of shares, on sliding and on full layers)
@pytest.mark.parametrize("geo", [(W.SLIDING, 256, 8, 2, 40), (W.SLIDING, 512, 4, 4, 33), (W.SLIDING, 64, 8, 1, 700),
                                 (W.FULL, 512, 8, 2, 0), (W.FULL, 128, 2, 2, 0)])
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
def test_steps_see_what_their_intervals_say(geo, dtype):
    L, window = 900, geo[4]
    lens = np.array([900, 31, 640, 500, 77, 1, 300])
    B = len(lens)
    at = lens - 1
    doc, span = np.zeros((B, L), int), np.full((B, L), -1)
    doc[0, 850:] = 1                       # a document that begins inside, one outside of a window of 40
    doc[2, 300:] = 1
    span[2, lens[2] - 20:lens[2]] = 3      # a token in a span that lies in the window
    span[3, 60:lens[3]] = 5                # and in one that begins before it
    doc[4, lens[4] - 1] = -1               # padding
    doc[6, lens[6] - 1] = 9                # a document of one token
    begin, end = i32(np.zeros((B, 1))), i32(np.zeros((B, 1)))
    G.g4_attn_visible_ranges(window, i32(at), i32(lens), i32(doc), i32(span), L, B, 1, begin, end)
    lo, hi = M.visible_ranges(window, at, lens, doc, span, L, 1)
    assert np.array_equal(begin.cpu().numpy(), lo) and np.array_equal(end.cpu().numpy(), hi)
    c = Case(geo, lens, L, dtype, 4)
    q = unit((B, 1, geo[2], geo[1]), 5, dtype)
    dq = q.to(DEV)
    pre = torch.full(q.shape, float("nan"), dtype=q.dtype, device=DEV)
    G.g4_attn_prefill_mods(c.params, c.table, 0, G.score_mods(20.0, None, begin, end), dq, i32(at), B, 1, pre)
    size = G.g4_attn_decode_mods_workspace_size(c.params, B, L)
    ws = torch.zeros(max(16, size), dtype=torch.uint8, device=DEV)
    dec = torch.full((B, geo[2], geo[1]), float("nan"), dtype=q.dtype, device=DEV)
    held = np.where(np.arange(B) == 4, 0, lens)   # (padding is a sequence that holds nothing)
    G.g4_attn_decode_mods(c.params, c.table, 0, G.score_mods(20.0, None, begin.view(B)), dq[:, 0].contiguous(), i32(held), B, L,
                          dec, ws, size)
    want, mass, mag = c.reference(f64(q), at[:, None], lo, hi, lens, 20.0, None)
    check(f64(pre), want, mass, mag, c.g, L, 20.0, dtype == W.BF16, ("prefill", geo))
    if 0 < window < lens[3] - 60:                 # the span's keys within the window
        lo = lo.copy()
        lo[3] = lens[3] - window
        want, mass, mag = c.reference(f64(q), at[:, None], lo, hi, lens, 20.0, None)
    check(f64(dec)[:, None], want, mass, mag, c.g, L, 20.0, False, ("decode", geo))
    assert (pre[4] == 0).all() and (dec[4] == 0).all()
    # the other way to say that a sequence sees nothing
    begin[4] = int(lens[4])
    G.g4_attn_decode_mods(c.params, c.table, 0, G.score_mods(20.0, None, begin.view(B)), dq[:, 0].contiguous(), i32(lens), B, L,
                          dec, ws, size)
    assert (dec[4] == 0).all()
