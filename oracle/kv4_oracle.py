"""Plain float64 CPU oracle of the paged 4-bit KV cache.

TEST INFRASTRUCTURE ONLY (as ``g4_oracle``): numpy in, numpy out, no code
shared with the CUDA library or the benchmark cases.

* ``quantise`` / ``values`` -- the numbers a row of bf16 values is held as:
  one e4m3 scale per 16 consecutive elements, s = RN(max |x| 2^-e / 6), and
  e2m1 codes RN(x 2^-e / s).
* ``record_offsets``  -- the byte order of a record, from the formulas of
  ``include/g4attn.h``.
* ``write_slot`` / ``read_rows`` -- rows into and out of a pool.
* ``assign_blocks``   -- block tables and slots by simulating a free list.
"""

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])  # e2m1 magnitudes
# e4m3 magnitudes by byte 0..126 (127 is NaN)
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])
NAN_SCALE = 127


def nearest(x, grid):
    """Index of the entry of the ascending ``grid`` nearest to x >= 0, ties to the even index."""
    dist = np.abs(x - grid)
    best = np.flatnonzero(dist == dist.min())
    return int(best[0]) if len(best) == 1 or best[0] % 2 == 0 else int(best[1])


def quantise(x, k_exp=0):
    """Codes (0..15) [..., hd] and scale bytes [..., hd/16] of rows x (float64 holding bf16 values).

    The scale's tie points times 6 and the codes' tie points times the scale
    are exact in float64, so the comparisons are made on products."""
    x = np.asarray(x, np.float64) * 2.0 ** -k_exp
    y = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    top = np.abs(y).max(-1)
    finite = np.isfinite(y).all(-1)
    mids = (E4M3[1:] + E4M3[:-1]) / 2 * 6
    t = np.where(finite, top, 0.0)
    up = np.searchsorted(mids, t, side="left")      # number of tie points below t
    tie = (up < len(mids)) & (mids[np.minimum(up, len(mids) - 1)] == t)
    scale = np.where(tie & (up % 2 == 1), up + 1, up)
    scale = np.where(finite, scale, NAN_SCALE).astype(np.uint8)
    s = np.where(finite, E4M3[np.minimum(scale, 126)], 0.0)[..., None]
    cm = (GRID[1:] + GRID[:-1]) / 2
    mag = np.zeros(y.shape, np.int64)
    ya = np.where(np.isfinite(y), np.abs(y), 0.0)
    for i in range(7):
        mag += ((ya > cm[i] * s) | ((ya == cm[i] * s) & (i % 2 == 1))) & (s > 0)
    code = mag + 8 * (np.signbit(y) & (s > 0))
    return code.reshape(x.shape).astype(np.uint8), scale


def values(code, scale, k_exp=0):
    """The numbers that codes and scale bytes stand for."""
    v = GRID[code & 7] * np.where(code >> 3, -1.0, 1.0)
    s = np.where(scale & 127 == NAN_SCALE, np.nan,  # (e4m3's 255 is a NaN too, though no quantiser writes it)
                 E4M3[np.minimum(scale & 127, 126)]) * np.where(scale >> 7, -1.0, 1.0)
    out = v.reshape(v.shape[:-1] + (-1, 16)) * s[..., None] * 2.0 ** k_exp
    return out.reshape(v.shape)


def record_offsets(hd):
    """Byte offsets in a record: (k code, k scale, v code, v scale), each [16 positions][hd] (codes: of the
    byte; the code of an even element is its low half)."""
    m = np.arange(16)[:, None]
    d = np.arange(hd)[None, :]
    p, w = d // 64, (d // 16) % 4
    r, g = m // 8, m % 8
    kc = 512 * p + 16 * (4 * g + (d % 16) // 4) + 8 * r + 2 * w + (d % 4) // 2
    ks = 8 * hd + 64 * p + 8 * g + 2 * w + r
    ih, t, il = m // 8, (m % 8) // 2, m % 2
    i = 2 * ih + il
    vc = 9 * hd + 512 * p + 16 * (4 * ((d % 16) // 2) + t) + 4 * i + w
    vs = 17 * hd + 64 * p + 16 * t + 4 * w + i
    return kc, ks, vc, vs


def write_slot(data, slot, kvh, k_row, v_row, block_size, k_exp=0):
    """Stores one position's rows (float64 holding bf16 values) at a slot of data [n_blocks, Hkv, bs/16, 18 hd]."""
    hd = k_row.shape[-1]
    rec = data[slot // block_size, kvh, (slot % block_size) // 16]
    m = slot % 16
    for off, soff, row, e in ((0, 1, k_row, k_exp), (2, 3, v_row, 0)):
        offs = record_offsets(hd)
        code, scale = quantise(row, e)
        rec[offs[off][m, 0::2]] = code[0::2] | (code[1::2] << 4)
        rec[offs[soff][m, 0::16]] = scale


def read_rows(data, table_row, kvh, positions, block_size, k_exp=0):
    """float64 K and V rows of ``positions``; NaN rows where the block id is outside the pool."""
    n_blocks, hd = data.shape[0], data.shape[-1] // 18
    kc, ks, vc, vs = record_offsets(hd)
    k, v = (np.full((len(positions), hd), np.nan) for _ in range(2))
    shift = 4 * (np.arange(hd) % 2)
    for n, p in enumerate(positions):
        e = p // block_size
        if p < 0 or e >= len(table_row) or not 0 <= table_row[e] < n_blocks:
            continue
        rec = data[table_row[e], kvh, (p % block_size) // 16]
        m = p % 16
        k[n] = values((rec[kc[m]] >> shift) & 15, rec[ks[m, 0::16]], k_exp)
        v[n] = values((rec[vc[m]] >> shift) & 15, rec[vs[m, 0::16]])
    return k, v


def assign_blocks(old, new, T, block_size, n_blocks, free, count, table):
    """Simulates one call: returns (table, free, count, lens, positions, slots); inputs are not changed.

    Entries given back that hold no block of the pool do not go onto the free list."""
    table, stack = np.array(table), [int(x) for x in free[:count]]
    free = np.array(free)
    B, width = table.shape
    ceil = lambda n: -(-n // block_size)  # noqa: E731
    cap = width * block_size
    old = [min(max(int(x), 0), cap) for x in old]
    new = [min(max(int(x), 0), cap, o + T) for x, o in zip(new, old)]
    for b in range(B):
        for e in range(ceil(new[b]), ceil(old[b])):
            if 0 <= table[b, e] < n_blocks:
                stack.append(int(table[b, e]))
    free[:len(stack)] = stack
    lens = list(old)
    refused = False
    for b in range(B):
        need = ceil(new[b]) - ceil(old[b])
        if need > 0:
            refused = refused or need > len(stack)
            if refused:
                continue
            for e in range(ceil(old[b]), ceil(new[b])):
                table[b, e] = stack.pop()
        lens[b] = new[b]
    positions, slots = np.full((B, T), -1), np.full((B, T), -1)
    for b in range(B):
        for t in range(min(T, lens[b] - old[b])):
            p = old[b] + t
            positions[b, t] = p
            i = table[b, p // block_size]
            slots[b, t] = i * block_size + p % block_size if 0 <= i < n_blocks else -1
    return table, free, len(stack), np.array(lens), positions, slots
