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
