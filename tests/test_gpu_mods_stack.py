"""AttnStack's calls with modified scores on streams of the caller's."""

import pytest

from gemma_dual_geometry_gb300 import build as g4build
from gemma_dual_geometry_gb300.stack import AttnStack
from gpu_common import DEV, G, W, torch
from test_gpu_mods import i32, unit

pytestmark = pytest.mark.gpu

CFG = dict(B=3, H=8, Hkv=2, dtype=W.BF16, seed=77, types=[W.SLIDING, W.FULL, W.SLIDING, W.FULL], n_shared=2,
           geom={W.SLIDING: dict(head_dim=64, theta=1e4, rotary_fraction=1.0, window=900),
                 W.FULL: dict(head_dim=128, theta=1e6, rotary_fraction=0.25, window=0)})


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    g4build.build()
    G.lib()
    yield
    assert G.g4_take_device_error() == 0


def inputs(st):
    """A query per layer, and caches that hold something."""
    qs = {}
    for l, g in enumerate(st.geo):
        qs[l] = unit((3, 8, g["head_dim"]), l, W.BF16).to(DEV)
        if st.owns(l):
            for i, c in enumerate(st.caches[l]):
                c.copy_(unit(tuple(c.shape), 10 * l + i, W.BF16))
    return qs


def test_a_stack_made_while_its_stream_is_busy():
    """The stack's memory is laid out on the current stream; what is called next may go to another one."""
    lens = i32([2000, 1500, 700])
    warm = AttnStack(CFG, 2000, device=DEV, mods=True)
    qs = inputs(warm)
    mods = G.score_mods(30.0)
    want = {l: torch.empty_like(q) for l, q in qs.items()}
    for l, q in qs.items():
        warm.decode_attn(l, q, lens, 2000, want[l], mods=mods)
    rows = {l: [c.clone() for c in kv] for l, kv in warm.caches.items()}
    sizes = [ws.numel() for ws in warm.mods_ws.values()]
    torch.cuda.synchronize()
    del warm
    # (the next stack's memory is this: counters that are not zero until it has been zero-filled)
    dirty = [torch.full((n,), 77, dtype=torch.uint8, device=DEV) for n in sizes]
    side = torch.cuda.Stream()
    out = {l: torch.empty_like(q) for l, q in qs.items()}
    torch.cuda.synchronize()
    del dirty
    torch.cuda._sleep(200_000_000)   # (about a tenth of a second on the current stream)
    st = AttnStack(CFG, 2000, device=DEV, mods=True)
    with torch.cuda.stream(side):
        for l, kv in rows.items():
            for c, r in zip(st.caches[l], kv):
                c.copy_(r)
        for l, q in qs.items():
            st.decode_attn(l, q, lens, 2000, out[l], mods=mods)
    torch.cuda.synchronize()
    for l in qs:
        assert torch.equal(out[l], want[l]), l


def test_layers_on_two_streams_at_once():
    """Decodes of two layers, each on a stream, give what they give one after another."""
    st = AttnStack(CFG, 2000, device=DEV, mods=True)
    qs = inputs(st)
    lens, mods = i32([2000, 1500, 700]), G.score_mods(30.0)
    want = {}
    for l, q in qs.items():
        want[l] = torch.empty_like(q)
        st.decode_attn(l, q, lens, 2000, want[l], mods=mods)
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [{l: torch.empty_like(q) for l, q in qs.items()} for _ in range(20)]
    torch.cuda.synchronize()
    for turn in outs:
        for l, q in qs.items():
            st.decode_attn(l, q, lens, 2000, turn[l], stream=streams[l], mods=mods)
    torch.cuda.synchronize()
    for turn in outs:
        for l in qs:
            assert torch.equal(turn[l], want[l]), l
