"""What the binding of the calls with modified scores and several axes refuses of its tensors and tables: kernels would
read past them, or at addresses that are not theirs (no GPU needed)."""

import pytest
import torch

from gemma_dual_geometry_gb300 import build as g4build
from gemma_dual_geometry_gb300 import g4attn as G

FAKE = 0x7f0000000000  # aligned, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _lib():
    g4build.build()
    G.lib()


class OnDevice:
    """A tensor of GPU ``index`` as far as the binding looks at it."""

    is_cuda = True

    def __init__(self, index, n=0, dtype=torch.int32):
        self.index, self.n, self.dtype = index, n, dtype

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def numel(self):
        return self.n

    def data_ptr(self):
        return FAKE


@pytest.fixture
def one_device(monkeypatch):
    monkeypatch.setattr(G, "_raw_stream", lambda device: 0, raising=False)
    monkeypatch.setattr(G, "_current_device", None, raising=False)


def params(**kw):
    return G.layer_params(**dict(dict(layer_type=G.G4_FULL, head_dim=64, n_heads=8, n_kv_heads=2), **kw))


def table():
    t = G.cache_table(1)
    G.set_cache(t, 0, FAKE, FAKE, G.G4_FULL, 64, 2, 100, 4, G.G4_BF16)
    return t


def prefill(mods, q=None, B=0, T=5):
    G.g4_attn_prefill_mods(params(), table(), 0, mods, q or OnDevice(0), FAKE, B, T, FAKE, 0)


def decode(mods, q=None, B=0):
    G.g4_attn_decode_mods(params(), table(), 0, mods, q or OnDevice(0), FAKE, B, 100, FAKE, FAKE, 1 << 30, 0)


def test_tensors_of_another_device_than_q(one_device):
    slopes, begin = OnDevice(0, 8, torch.float32), OnDevice(0, 100)
    for call in (prefill, decode):
        call(G.score_mods(30.0, slopes, begin))
        call(G.score_mods(30.0, slopes, begin), FAKE)
        call(G.score_mods(30.0, FAKE, FAKE))
        call(None)
        for mods in (G.score_mods(0.0, torch.ones(8)), G.score_mods(0.0, None, torch.zeros(100, dtype=torch.int32))):
            with pytest.raises(ValueError, match="device"):   # the host's, whatever q is
                call(mods)
            with pytest.raises(ValueError, match="device"):
                call(mods, FAKE)
        with pytest.raises(ValueError, match="device"):
            call(G.score_mods(0.0, slopes), OnDevice(1))
    for pair in ((slopes, OnDevice(1, 100)), (torch.ones(8), begin)):
        with pytest.raises(ValueError, match="devices"):
            G.score_mods(0.0, *pair)


def test_fewer_entries_than_heads_or_tokens(one_device):
    def slopes(n):
        return G.score_mods(0.0, OnDevice(0, n, torch.float32))

    for call in (prefill, decode):
        call(slopes(8))
        call(slopes(9))
        for n in (0, 2, 7):   # (2: a slope for each kv head)
            with pytest.raises(ValueError, match="8 entries"):
                call(slopes(n))
    # (nothing is launched: the workspace is too small, T exceeds the cache)
    for n, T, refused in ((4 * 101, 101, False), (4 * 101 - 1, 101, True), (4, 101, True)):
        for given in ((OnDevice(0, n), None), (OnDevice(0, n), OnDevice(0, 4 * 101)), (FAKE, OnDevice(0, n))):
            with pytest.raises(ValueError if refused else G.G4Error):
                prefill(G.score_mods(0.0, None, *given), B=4, T=T)
    for n, refused in ((4, False), (3, True)):
        with pytest.raises(ValueError if refused else G.G4Error):
            G.g4_attn_decode_mods(params(), table(), 0, G.score_mods(0.0, None, OnDevice(0, n)), OnDevice(0), FAKE, 4, 100,
                                  FAKE, FAKE, 0, 0)


@pytest.mark.parametrize("axis", [[0, 256], [0, -1], [0, 0.5], [0, 300.0], [float("nan")]])
def test_axes_that_a_byte_does_not_hold(axis):
    """(256 became axis 0, -1 axis 255.)"""
    with pytest.raises(ValueError, match="whole numbers"):
        G.rope_axes(2, axis, 64)


def test_tables_that_stop_short_of_the_rotated_pairs():
    """(The rest were turned by axis 0, or by no angle at all; tables of a smaller head were read past their end.)"""
    def call(axes, **kw):
        p = params(**kw)
        t = G.cache_table(1)
        G.set_cache(t, 0, FAKE, FAKE, G.G4_FULL, p.head_dim, 2, 100, 4, G.G4_BF16)
        G.g4_kv_append_normrope_axes(p, t, 0, axes, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, 5, FAKE, 0)

    call(G.rope_axes(2, [0, 1] * 16, 64))
    call(G.rope_axes(2, [0, 1] * 4, 64), rotary_fraction=0.25)
    call(G.rope_axes(2, [0, 1] * 4, 64, [0.5] * 8), rotary_fraction=0.25)
    call(G.rope_axes(2, [0, 1] * 16, 64), head_dim=128, rotary_fraction=0.5)
    call(G.rope_axes(1, [], 64), rotary_fraction=0.0)
    for axes, kw in ((G.rope_axes(2, [0, 1] * 15 + [0], 64), {}), (G.rope_axes(2, [0, 1] * 16, 64, [0.5] * 31), {}),
                     (G.rope_axes(2, [0, 1] * 3, 64), dict(rotary_fraction=0.25)),
                     (G.rope_axes(2, [0, 1] * 4, 64, [0.5] * 7), dict(rotary_fraction=0.25)),
                     (G.rope_axes(2, [0, 1] * 16, 64), dict(head_dim=128)), (G.rope_axes(1, [], 64), {})):
        with pytest.raises(ValueError, match="pairs"):
            call(axes, **kw)


def refused(fn, *args):
    with pytest.raises(G.G4Error) as e:
        fn(*args)
    return e.value.status == G.G4_ERR_INVALID_ARG and "4-byte aligned" in str(e.value)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_arrays_that_are_not_aligned(off):
    """Positions, lengths, ids and intervals are 32-bit numbers: at other addresses their loads fault."""
    odd = FAKE + off
    for i in (1, 2, 3, 4, 8, 9):
        args = [0, FAKE, FAKE, FAKE, FAKE, 10, 1, 0, FAKE, FAKE, 0]
        G.g4_attn_visible_ranges(*args)
        args[i] = odd
        assert refused(G.g4_attn_visible_ranges, *args), i
    axes = G.rope_axes(1, [0] * 32, 64)
    for i in (9, 10):
        args = [params(), table(), 0, axes, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, 0, FAKE, 0]
        G.g4_kv_append_normrope_axes(*args)
        args[i] = odd
        assert refused(G.g4_kv_append_normrope_axes, *args), i
    assert refused(G.g4_attn_prefill_mods, params(), table(), 0, None, FAKE, odd, 1, 0, FAKE, 0)
    assert refused(G.g4_attn_decode_mods, params(), table(), 0, None, FAKE, odd, 0, 100, FAKE, FAKE, 1 << 30, 0)
