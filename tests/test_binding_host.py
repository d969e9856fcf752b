"""What the Python binding takes for a pointer, and refuses (no GPU needed)."""

import numpy as np
import pytest
import torch

from gemma_dual_geometry_gb300 import g4attn as G


@pytest.mark.parametrize("x", [b"\0" * 64, "q", 1.5, [1, 2], np.zeros(4, np.int32), object()])
def test_only_tensors_addresses_and_none_are_pointers(x):
    """Anything else raises before the library is called: ctypes would take bytes and strings for addresses."""
    with pytest.raises(AttributeError):
        G._ptr(x)
    table = G.kv4_pool_table(1)
    with pytest.raises(AttributeError):
        G.set_kv4_pool(table, 0, x, G.G4_FULL, 64, 1, 1, 16)


def test_tensors_addresses_and_none():
    t = torch.zeros(4)
    assert G._ptr(t) == t.data_ptr() and G._ptr(4096) == 4096 and G._ptr(None) is None


class OnDevice:
    """A tensor of GPU ``index`` as far as the binding looks at it."""

    is_cuda = True

    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 0x7f0000000000


class Stream:
    def __init__(self, raw):
        self.cuda_stream = raw


def test_tensors_of_another_device_than_the_current_one(monkeypatch):
    """A launch goes to the current device, and every device's default stream has the address 0: tensors of another
    device are refused there.  (A stream of its own that belongs to another device is the launch's error.)"""
    monkeypatch.setattr(G, "_raw_stream", lambda device: 0, raising=False)
    monkeypatch.setattr(G, "_current_device", lambda: 1, raising=False)
    p = G.layer_params(G.G4_FULL, 64, 2, 2)
    pools = G.kv4_pool_table(1)

    def gather(index, **kw):   # (no rows: nothing is launched)
        t = OnDevice(index)
        G.set_kv4_pool(pools, 0, t, G.G4_FULL, 64, 2, 4, 16)
        G.g4_kv4_gather(p, pools, 0, t, 4, t, t, 1, 0, t, t, **kw)

    gather(1)
    gather(1, stream=Stream(0))
    gather(0, stream=Stream(0x1000))
    for kw in ({}, dict(stream=0), dict(stream=Stream(0))):
        with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
            gather(0, **kw)
    monkeypatch.setattr(G, "_current_device", None, raising=False)   # the only device there is
    gather(0)
