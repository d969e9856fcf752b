"""float64 oracle of attention with modified scores, of the intervals of keys and of the append with several axes.

Numpy, from the definitions in include/g4attn.h; it shares no code with the kernels or with the benchmark's cases.
"""

import numpy as np

from oracle import g4_oracle as O


def visible_ranges(window, q_start, seq_lens, doc_ids, span_ids, max_len, T):
    """(key_begin, key_end) [B, T] of tokens at positions q_start[b] + t: what each sees, token by token."""
    B = len(q_start)
    begin, end = np.zeros((B, T), np.int64), np.zeros((B, T), np.int64)
    for b in range(B):
        held = min(max(int(seq_lens[b]), 0), max_len)
        doc = [0] * held if doc_ids is None else [int(x) for x in doc_ids[b][:held]]
        span = [-1] * held if span_ids is None else [int(x) for x in span_ids[b][:held]]
        first_of_doc, first_of_span, end_of_span = [0] * held, [0] * held, [0] * held
        for p in range(held):
            new_doc = p == 0 or doc[p] != doc[p - 1]
            first_of_doc[p] = p if new_doc else first_of_doc[p - 1]
            first_of_span[p] = p if new_doc or span[p] != span[p - 1] else first_of_span[p - 1]
        for p in reversed(range(held)):
            same = p + 1 < held and first_of_span[p + 1] == first_of_span[p]
            end_of_span[p] = end_of_span[p + 1] if same else p + 1
        for t in range(T):
            p = int(q_start[b]) + t
            if p < 0 or p >= held or doc[p] < 0:
                continue
            begin[b, t] = max(first_of_doc[p], p - window + 1) if window > 0 else first_of_doc[p]
            end[b, t] = p + 1
            if span[p] >= 0:
                begin[b, t] = min(begin[b, t], first_of_span[p])
                end[b, t] = end_of_span[p]
    return begin, end


def modified(s, distance, cap, slope):
    """Scores s with a cap (0: none) and a bias of slope (0: none) times the distance."""
    if cap:
        s = cap * np.tanh(s / cap)
    return s - slope * np.abs(distance)


def attention_rows(q, k, v, k_pos, q_pos, begin, end, cap=0.0, slope=0.0, scale=1.0):
    """One head: q [T, hd] at positions q_pos against keys k, v [n, hd] at positions k_pos; query t sees begin[t] <=
    k_pos < end[t].  Returns (output [T, hd], sum_j p_j |v_j|, the largest sum_d |q_d k_d| scale + |bias| of a key that
    t sees [T]).  Rows of keys that nobody sees may hold anything."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    sees = (k_pos[None, :] >= np.asarray(begin)[:, None]) & (k_pos[None, :] < np.asarray(end)[:, None])
    used = sees.any(0)
    k, v, k_pos, sees = k[used], v[used], k_pos[used], sees[:, used]
    out, mass = np.zeros((len(q), v.shape[1])), np.zeros((len(q), v.shape[1]))
    size = np.zeros(len(q))
    if not used.any():
        return out, mass, size
    distance = np.asarray(q_pos)[:, None] - k_pos[None, :]
    s = modified((q @ k.T) * scale, distance, cap, slope)
    s = np.where(sees, s, -np.inf)
    top = s.max(1, keepdims=True)
    p = np.where(sees, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
    total = p.sum(1, keepdims=True)
    p = p / np.where(total > 0, total, 1.0)
    size = np.where(sees, (np.abs(q) @ np.abs(k).T) * scale + np.abs(slope * distance), 0.0).max(1)
    return p @ v, p @ np.abs(v), size


def default_intervals(q_pos, layer_type, window):
    """What the tokens at q_pos see without intervals of their own."""
    q_pos = np.asarray(q_pos, np.int64)
    begin = np.maximum(0, q_pos - window + 1) if layer_type == O.SLIDING else np.zeros_like(q_pos)
    return begin, q_pos + 1


def rope_axes(x, positions, axis, inv_freq):
    """rotate_half RoPE of rows x [..., heads, hd] whose pair j is turned by positions[axis[j]] [n_axes, ...]."""
    half = x.shape[-1] // 2
    f = np.asarray(inv_freq, np.float32).astype(np.float64)
    pos = np.asarray(positions, np.float64)
    angle = np.stack([pos[axis[j] if j < len(axis) else 0] * f[j] for j in range(half)], -1)[..., None, :]
    a, b = x[..., :half], x[..., half:]
    return np.concatenate([a * np.cos(angle) - b * np.sin(angle), b * np.cos(angle) + a * np.sin(angle)], -1)


def normrope_axes(x, w, positions, axis, inv_freq, eps):
    """Normed and roped rows, float64."""
    return rope_axes(O.rms_norm(x, w, eps), positions, axis, inv_freq)
