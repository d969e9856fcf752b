"""Pins of the 4-bit cache's oracle (no GPU): its rounding against a search
over all representable numbers and torch's own e4m3 cast, its byte order
against the properties a layout must have, its block assignment against
conservation of blocks."""

import numpy as np
import pytest
import torch

from oracle import g4_oracle as O
from oracle import kv4_oracle as K


def test_e4m3_table_is_torchs():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(K.E4M3, t)


def test_codes_are_the_nearest_by_search():
    rng = np.random.default_rng(0)
    x = O.round_bf16(rng.standard_normal((40, 64)) * np.exp(rng.uniform(-6, 6, (40, 1))))
    x[3] = 0.0
    x[4, :16] = 2.0 ** -12      # scale underflows to the smallest e4m3, or to zero
    x[5, 16:32] = 5000.0        # saturates
    code, scale = K.quantise(x)
    for i in range(x.shape[0]):
        for blk in range(4):
            y = np.abs(x[i, 16 * blk:16 * blk + 16])
            assert scale[i, blk] == K.nearest(y.max() / 6, K.E4M3)
            s = K.E4M3[scale[i, blk]]
            for d in range(16):
                c = code[i, 16 * blk + d]
                assert (c & 7) == (K.nearest(y[d] / s, K.GRID) if s > 0 else 0)


def test_ties_go_to_even():
    # scale 1 (max 6): the tie points of e2m1
    row = np.array([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] + [-0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0])
    code, scale = K.quantise(row[None])
    assert K.values(code, scale)[0].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, -6]
    # tie points of the scale: max = 6 (1 + 1/16) lies between 1 and 1.125
    for top, want in ((6 * 1.0625, 1.0), (6 * 1.1875, 1.25)):
        assert K.E4M3[K.quantise(np.full((1, 16), top))[1][0, 0]] == want


def test_values_fit_bf16_and_error_is_bounded():
    rng = np.random.default_rng(1)
    x = O.round_bf16(rng.standard_normal((64, 128)))
    for e in (0, -3, 5):
        v = K.values(*K.quantise(x, e), e)
        assert np.array_equal(O.round_bf16(v), v)
    # half a step of e2m1 next to 6 is 1 of 6, of a scale that is off by 2^-4 at most
    v = K.values(*K.quantise(x))
    top = np.abs(x.reshape(64, 8, 16)).max(-1, keepdims=True)
    assert (np.abs(v - x).reshape(64, 8, 16) <= top * (1 / 6 + 2.0 ** -4 + 0.01)).all()


def test_power_of_two_exponent_shifts_the_values():
    rng = np.random.default_rng(2)
    x = O.round_bf16(rng.standard_normal((8, 64)))
    a, b = K.quantise(x), K.quantise(x * 2.0 ** -7, -7)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_non_finite_blocks_stand_for_nans():
    x = np.ones((3, 32))
    x[0, 5], x[1, 20] = np.nan, np.inf
    v = K.values(*K.quantise(x))
    assert np.isnan(v[0, :16][np.array(K.quantise(x)[0][0, :16]) > 0]).all() and np.isfinite(v[0, 16:]).all()
    assert np.isfinite(v[1, :16]).all() and K.quantise(x)[1][1, 1] == K.NAN_SCALE
    assert np.isfinite(v[2]).all()


@pytest.mark.parametrize("hd", [64, 128, 256, 512])
def test_record_bytes_are_used_once(hd):
    kc, ks, vc, vs = K.record_offsets(hd)
    used = np.concatenate([kc[:, 0::2].ravel(), ks[:, 0::16].ravel(), vc[:, 0::2].ravel(), vs[:, 0::16].ravel()])
    assert sorted(used) == list(range(18 * hd))
    # both elements of a byte, and all of a block's scale, agree on it
    for o, step in ((kc, 2), (vc, 2), (ks, 16), (vs, 16)):
        for i in range(1, step):
            assert np.array_equal(o[:, 0::step], o[:, i::step])


def test_write_then_read():
    rng = np.random.default_rng(3)
    data = rng.integers(0, 256, (3, 2, 2, 18 * 64), dtype=np.uint8)
    before = data.copy()
    rows = O.round_bf16(rng.standard_normal((2, 64)))
    K.write_slot(data, 2 * 32 + 21, 1, rows[0], rows[1], 32, k_exp=1)
    k, v = K.read_rows(data, [7, 2], 1, [32 + 21, 0], 32, k_exp=1)
    assert np.array_equal(k[0], K.values(*K.quantise(rows[0], 1), 1)) and np.isnan(k[1]).all()
    assert np.array_equal(v[0], K.values(*K.quantise(rows[1])))
    changed = np.argwhere(data != before)
    assert len(changed) <= 2 * (32 + 4) and {tuple(c[:3]) for c in changed} == {(2, 1, 1)}


def test_assign_conserves_blocks():
    rng = np.random.default_rng(4)
    B, width, bs, n = 13, 6, 16, 50
    table, free = np.full((B, width), -1), rng.permutation(n)
    count, lens = n, np.zeros(B, int)
    for step in range(60):
        T = int(rng.integers(1, 40))
        new = np.where(rng.random(B) < 0.3, 0, np.minimum(lens + rng.integers(0, T + 1, B), width * bs))
        table, free, count, got, pos, slots = K.assign_blocks(lens, new, T, bs, n, free, count, table)
        assert all(g in (o, w) for g, o, w in zip(got, lens, new))
        held = [int(table[b, e]) for b in range(B) for e in range(-(-got[b] // bs))]
        everything = held + [int(x) for x in free[:count]]
        assert sorted(everything) == list(range(n))
        flat = slots[slots >= 0]
        assert len(set(flat.tolist())) == len(flat)
        lens = got
