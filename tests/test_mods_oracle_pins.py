"""Pins of oracle/mods_oracle.py: against other forms of the same definitions (no GPU needed)."""

import numpy as np
import pytest
import torch

from oracle import g4_oracle as O
from oracle import mods_oracle as M


def pairwise(window, doc, span, held, p, j):
    """Whether position p sees position j, from the ids between them alone."""
    if not (0 <= p < held and 0 <= j < held) or doc[p] < 0:
        return False
    lo, hi = min(p, j), max(p, j)
    one_doc = len(set(doc[lo:hi + 1])) == 1
    one_span = one_doc and span[p] >= 0 and len(set(span[lo:hi + 1])) == 1
    return one_span or (one_doc and j <= p and (window == 0 or p - j < window))


@pytest.mark.parametrize("window", [0, 1, 4, 100])
def test_intervals_are_the_pairs_that_ids_allow(window):
    rng = np.random.default_rng(window)
    for _ in range(30):
        L = int(rng.integers(1, 40))
        doc = np.repeat(rng.integers(-1, 3, L), rng.integers(1, 9, L))[:L]
        span = np.repeat(rng.integers(-2, 3, L), rng.integers(1, 6, L))[:L]
        held = int(rng.integers(0, L + 1))
        start = int(rng.integers(-3, L + 1))
        T = int(rng.integers(1, 45))
        begin, end = M.visible_ranges(window, [start], [held], [doc], [span], L, T)
        for t in range(T):
            p = start + t
            sees = [j for j in range(L) if pairwise(window, list(doc), list(span), held, p, j)]
            assert list(range(begin[0, t], end[0, t])) == sees, (p, doc, span, held)


def test_whole_rows():
    """Without ids: the causal intervals; all one span: every token sees all."""
    b, e = M.visible_ranges(0, [0], [9], None, None, 9, 9)
    assert b.tolist() == [[0] * 9] and e.tolist() == [list(range(1, 10))]
    b, e = M.visible_ranges(3, [0], [9], None, [[5] * 9], 9, 9)
    assert b.tolist() == [[0] * 9] and e.tolist() == [[9] * 9]
    b, e = M.visible_ranges(3, [4], [9], None, None, 9, 6)
    assert b.tolist() == [[2, 3, 4, 5, 6, 0]] and e.tolist() == [[5, 6, 7, 8, 9, 0]]


def test_attention_without_modifications_is_the_paths():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((1, 7, 1, 16)), rng.standard_normal((1, 1, 7, 16)), rng.standard_normal((1, 1, 7, 16))
    for lt, w in ((O.SLIDING, 3), (O.FULL, 0)):
        want = O.attention(q, k, v, np.arange(7)[None], [7], 1, lt, w)
        begin, end = M.default_intervals(np.arange(7), lt, w)
        got, _, _ = M.attention_rows(q[0, :, 0], k[0, 0], v[0, 0], np.arange(7), np.arange(7), begin, end)
        np.testing.assert_allclose(got, want[0, :, 0], rtol=0, atol=1e-12)


def test_caps_and_biases_against_torch():
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal((11, 32)) * 3 for _ in range(3))
    at = np.arange(11)
    begin, end = rng.integers(0, 6, 11), rng.integers(4, 12, 11)
    got, mass, size = M.attention_rows(q, k, v, at, at, begin, end, cap=5.0, slope=0.25, scale=0.5)
    s = torch.tanh(torch.tensor(q @ k.T) * 0.5 / 5.0) * 5.0 - 0.25 * (torch.tensor(at)[:, None] - torch.tensor(at)).abs()
    hidden = torch.tensor((at[None] < begin[:, None]) | (at[None] >= end[:, None]))
    p = torch.softmax(s.masked_fill(hidden, -np.inf), 1).nan_to_num()
    np.testing.assert_allclose(got, p @ torch.tensor(v), atol=1e-12)
    np.testing.assert_allclose(mass, p @ torch.tensor(np.abs(v)), atol=1e-12)
    assert (size > 0).all() == (begin < end).all()
    # a cap far above the scores changes nothing, one far below makes all keys equal
    free, _, _ = M.attention_rows(q, k, v, at, at, begin * 0, end * 0 + 11)
    np.testing.assert_allclose(M.attention_rows(q, k, v, at, at, begin * 0, end * 0 + 11, cap=1e9)[0], free, atol=1e-9)
    np.testing.assert_allclose(M.attention_rows(q, k, v, at, at, begin * 0, end * 0 + 11, cap=1e-9)[0],
                               np.repeat(v.mean(0)[None], 11, 0), atol=1e-6)


def test_rows_that_see_nothing_and_keys_that_nobody_sees():
    q, k = np.ones((2, 4)), np.ones((3, 4))
    v = np.array([[np.nan] * 4, [2.0] * 4, [np.inf] * 4])
    out, mass, _ = M.attention_rows(q, k, v, np.arange(3), np.arange(2), [1, 2], [2, 2])
    assert out.tolist() == [[2.0] * 4, [0.0] * 4] and mass.tolist() == [[2.0] * 4, [0.0] * 4]


def test_axes_that_agree_are_one_position():
    rng = np.random.default_rng(2)
    x, pos = rng.standard_normal((2, 5, 3, 32)), rng.integers(0, 1000, (2, 5))
    inv = O.rope_inv_freq(32, 1e4, 0.5)
    want = O.rope_rotate_half(x, pos[..., None], inv)
    np.testing.assert_array_equal(M.rope_axes(x, np.stack([pos] * 3), [0, 2, 1, 1, 0, 2, 0, 1], inv), want)
    # an axis turns its own pairs only: complex form, pair by pair
    poss = rng.integers(0, 1000, (3, 2, 5))
    axis = [j % 3 for j in range(8)]
    got = M.rope_axes(x, poss, axis, inv)
    for j in range(16):
        z = x[..., j] + 1j * x[..., j + 16]
        if j < 8:
            z = z * np.exp(1j * poss[axis[j]] * np.float64(inv[j]))[..., None]
        np.testing.assert_allclose(got[..., j] + 1j * got[..., j + 16], z, atol=1e-12)
