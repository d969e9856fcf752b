"""What PagedAttnStack holds and hands to the library's calls, on the host: the calls that launch are replaced by
ones that note their arguments (no GPU needed)."""

import pytest
import torch

from gemma_dual_geometry_gb300 import build as g4build
from gemma_dual_geometry_gb300 import g4attn as G
from gemma_dual_geometry_gb300 import stack as S
from gemma_dual_geometry_gb300 import workloads as W

CFG = dict(B=3, H=4, Hkv=2, dtype=W.BF16, seed=0, types=[W.SLIDING, W.FULL, W.SLIDING, W.FULL], n_shared=2,
           geom={W.SLIDING: dict(head_dim=64, theta=1e4, rotary_fraction=1.0, window=24),
                 W.FULL: dict(head_dim=128, theta=1e6, rotary_fraction=0.25, window=0)})


@pytest.fixture
def calls(monkeypatch):
    """(name, arguments by position) of the calls made."""
    g4build.build()
    G.lib()
    seen = []
    for name in ("g4_kv4_assign_blocks", "g4_kv4_append_normrope", "g4_kv4_attn_prefill", "g4_kv4_attn_decode"):
        monkeypatch.setattr(G, name, lambda *a, stream=None, name=name: seen.append((name, a)))
    return seen


def make(**kw):
    return S.PagedAttnStack(CFG, max_len=160, n_blocks=26, block_size=32, device="cpu", **kw)


def lens(*x):
    return torch.tensor(x, dtype=torch.int32)


def prefill(st, T, calls, l=1):
    q = torch.zeros((3, T, 4, 128), dtype=torch.bfloat16)
    st.prefill_attn(l, q, T, q)
    name, a = calls[-1]
    assert name == "g4_kv4_attn_prefill"
    return a[-2], a[-1]   # workspace and its bytes


def need(st, T, l=1):
    return G.g4_kv4_prefill_workspace_size(st.params[l], 3, T, st.max_len)


@pytest.mark.parametrize("T", [1, 2, 40])
def test_prefill_has_the_workspace_it_needs(calls, T):
    """A prompt of one token too."""
    st = make()
    st.assign(lens(T, T, T), T)
    ws, size = prefill(st, T, calls)
    assert size >= need(st, T) > 0 and ws.numel() >= size


def test_decode_steps_hold_no_prefill_workspace(calls):
    st = make()
    before = held(st)
    st.assign(lens(1, 1, 1), 1)
    q = torch.zeros((3, 4, 128), dtype=torch.bfloat16)
    st.decode_attn(1, q, q)
    assert held(st) - before <= 2 * 4 * 3 + 64


def held(st):
    """Bytes of the tensors that an object keeps, in containers too."""
    found = {}

    def look(x):
        if isinstance(x, torch.Tensor):
            found[x.data_ptr()] = x.untyped_storage().nbytes()
        elif isinstance(x, dict):
            for y in x.values():
                look(y)
        elif isinstance(x, (list, tuple, set)):
            for y in x:
                look(y)

    look(vars(st))
    return sum(found.values())


def test_prefills_share_one_workspace(calls):
    """Chunks of any lengths: what is held is the longest one's, not one per length."""
    st = make()
    before = held(st)
    order = [40, 2, 39, 1, 17, 80] + list(range(3, 60))
    for T in order:
        st.assign(lens(T, T, T), T)
        for l in range(4):
            ws, size = prefill(st, T, calls, l)
            assert size >= max(need(st, T, i) for i in range(4)) and ws.numel() >= size
    small = sum(2 * 4 * 3 * T for T in set(order))   # positions and slots
    assert held(st) - before <= max(need(st, 80, i) for i in range(4)) + small


def test_a_captured_workspace_outlives_a_larger_one(calls, monkeypatch):
    """A graph goes on using the workspace that it was captured with."""
    st = make()
    monkeypatch.setattr(st, "_capturing", lambda stream: True)
    first, size = prefill(st, 5, calls)
    monkeypatch.setattr(st, "_capturing", lambda stream: False)
    at = first.data_ptr()
    del first
    calls.clear()
    prefill(st, 60, calls)
    prefill(st, 70, calls)   # (not captured: replaced)
    calls.clear()
    kept = []
    for x in vars(st).values():
        kept += [y for y in (x if isinstance(x, list) else [x]) if isinstance(y, torch.Tensor)]
    assert at in [x.data_ptr() for x in kept]
    assert held(st) >= size + need(st, 70)
    assert sum(x.untyped_storage().nbytes() == need(st, 60) for x in kept) == 0


@pytest.mark.parametrize("want", [[4, 4, 4], torch.tensor([4, 4, 4]), torch.tensor([4.0, 4.0, 4.0]), lens(4, 4), lens(4, 4, 4, 4),
                                  lens(4, 0, 4, 0, 4, 0)[::2], None])
def test_assign_takes_int32_lengths_of_its_sequences_only(calls, want):
    """64-bit lengths, read as 32-bit ones, would end sequences."""
    st = make()
    with pytest.raises(ValueError, match="new_lens"):
        st.assign(want, 4)
    assert not calls and not st._steps
    st.assign(lens(4, 4, 4), 4)
    st.assign(lens(8, 8, 8).data_ptr(), 4)   # an address is the caller's word
    assert len(calls) == 2


def test_append_follows_an_assignment(calls):
    """Before one of as many tokens there are no slots: the rows of all tokens would go to slot 0."""
    st = make()
    x = [torch.zeros((3, 4, n, 128), dtype=torch.bfloat16) for n in (4, 2, 2)]
    w = torch.zeros(128)
    st.assign(lens(1, 1, 1), 1)
    calls.clear()
    with pytest.raises(ValueError, match="assign"):
        st.append(1, *x, w, w, 4, torch.empty_like(x[0]))
    assert not calls
    st.assign(lens(5, 5, 5), 4)
    st.append(1, *x, w, w, 4, torch.empty_like(x[0]))
    assert calls[-1][0] == "g4_kv4_append_normrope"


def test_prefills_of_no_or_too_many_tokens_leave_the_workspace(calls):
    """No tokens need none; more than fit a sequence are the call's to refuse, and those after it find what they need."""
    st = make()
    ws, size = prefill(st, 0, calls)
    assert size == ws.numel() == 0
    prefill(st, 9, calls)
    before = held(st)
    prefill(st, st.max_len + 1, calls)
    assert held(st) == before
    prefill(st, 0, calls)
    for T in (5, 9, 30, st.max_len):
        ws, size = prefill(st, T, calls)
        assert ws.numel() >= size >= need(st, T)


def test_an_outgrown_workspace_of_a_stream_known_by_address(calls, monkeypatch):
    """Nothing tells when such a stream is done with it: it goes after the device has caught up, or not at all
    while a capture forbids waiting."""
    st = make()
    waits = []
    monkeypatch.setattr(st, "_wait_for_all", lambda: waits.append(st._prefill_T))
    q = torch.zeros((3, 90, 4, 128), dtype=torch.bfloat16)
    for T in (5, 7):
        st.prefill_attn(1, q[:, :T], T, q[:, :T])
    assert not waits
    st.prefill_attn(1, q[:, :5], 5, q[:, :5], stream=0x1000)
    st.prefill_attn(1, q[:, :30], 30, q[:, :30])
    assert waits == [7]
    monkeypatch.setattr(st, "_capturing", lambda stream: True)
    ws, _ = prefill(st, 40, calls)
    assert waits == [7] and len(st._kept_ws) == 1 and st._kept_ws[0].data_ptr() != ws.data_ptr()
