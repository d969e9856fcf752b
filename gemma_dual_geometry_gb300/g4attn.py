"""ctypes binding of libg4attn.so (declared in include/g4attn.h).

Argument marshalling only: every step of the attention path runs in the CUDA
kernels behind the C ABI.  Tensor arguments may be torch tensors (their
``data_ptr()`` is passed) or raw integer device addresses.  The functions
keep the C names; a non-OK status raises ``G4Error`` with the library's
message.  There is no fallback: if the library is not built, ``lib()``
raises.
"""

from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libg4attn.so")

G4_OK, G4_ERR_INVALID_ARG, G4_ERR_UNSUPPORTED, G4_ERR_SHARE_MISMATCH = 0, 1, 2, 3
G4_ERR_CAPACITY, G4_ERR_WORKSPACE, G4_ERR_CUDA = 4, 5, 6
G4_SLIDING, G4_FULL = 0, 1
G4_F32, G4_BF16 = 0, 1

STATUS_NAMES = {0: "G4_OK", 1: "G4_ERR_INVALID_ARG", 2: "G4_ERR_UNSUPPORTED", 3: "G4_ERR_SHARE_MISMATCH",
                4: "G4_ERR_CAPACITY", 5: "G4_ERR_WORKSPACE", 6: "G4_ERR_CUDA"}

_c_void_p = ctypes.c_void_p
_i32 = ctypes.c_int32


class G4LayerParams(ctypes.Structure):
    _fields_ = [("layer_type", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("window", ctypes.c_int32), ("theta", ctypes.c_float),
                ("rotary_fraction", ctypes.c_float), ("eps", ctypes.c_float), ("attn_scale", ctypes.c_float),
                ("kv_share_src", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class G4KVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("layer_type", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("max_len", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("dtype", ctypes.c_int32), ("ring", ctypes.c_int32)]


class G4KV4Pool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("layer_type", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("n_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("k_exp", ctypes.c_int32)]


class G4ScoreMods(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("key_begin", ctypes.c_void_p),
                ("key_end", ctypes.c_void_p)]


class G4RopeAxes(ctypes.Structure):
    _fields_ = [("n_axes", ctypes.c_int32), ("axis", ctypes.POINTER(ctypes.c_uint8)),
                ("inv_freq", ctypes.POINTER(ctypes.c_float))]


_P = ctypes.POINTER
# Every function include/g4attn.h declares, with its ctypes signature.
SIGNATURES = {
    "g4_kv_share_src": (_i32, [_i32, _i32, _P(_i32), _i32]),
    "g4_kv_append_normrope": (_i32, [_P(G4LayerParams), _P(G4KVCache), _i32, _i32, _c_void_p, _c_void_p, _c_void_p,
                                     _c_void_p, _c_void_p, _c_void_p, _i32, _i32, _c_void_p, _c_void_p]),
    "g4_attn_prefill": (_i32, [_P(G4LayerParams), _P(G4KVCache), _i32, _i32, _c_void_p, _c_void_p, _i32, _i32,
                               _c_void_p, _c_void_p]),
    "g4_attn_encoder": (_i32, [_P(G4LayerParams), _P(G4KVCache), _i32, _i32, _c_void_p, _i32, _i32, _c_void_p,
                               _c_void_p]),
    "g4_attn_decode_workspace_size": (ctypes.c_size_t, [_P(G4LayerParams), _i32, _i32]),
    "g4_attn_decode": (_i32, [_P(G4LayerParams), _P(G4KVCache), _i32, _i32, _c_void_p, _c_void_p, _i32, _i32,
                              _c_void_p, _c_void_p, ctypes.c_size_t, _c_void_p]),
    "g4_decode_step": (_i32, [_P(G4LayerParams), _P(G4KVCache), _i32, _i32, _c_void_p, _c_void_p, _c_void_p,
                              _c_void_p, _c_void_p, _c_void_p, _i32, _i32, _c_void_p, _c_void_p, ctypes.c_size_t,
                              _c_void_p]),
    "g4_attn_decode_noalloc": (_i32, [_P(G4LayerParams), _P(G4KVCache), _i32, _i32, _c_void_p, _c_void_p, _i32,
                                      _i32, _c_void_p, _c_void_p]),
    "g4_qkv_project_append": (_i32, [_P(G4LayerParams), _P(G4KVCache), _i32, _i32, _c_void_p, _i32, _c_void_p,
                                     _c_void_p, _c_void_p, _c_void_p, _i32, _i32, _c_void_p, _c_void_p]),
    "g4_attn_out_residual": (_i32, [_c_void_p, _i32, _i32, _c_void_p, _i32, _c_void_p, ctypes.c_float, _c_void_p,
                                    _c_void_p, _c_void_p]),
    "g4_kv4_assign_blocks": (_i32, [_i32] * 5 + [_c_void_p] * 10),
    "g4_kv4_append_normrope": (_i32, [_P(G4LayerParams), _P(G4KV4Pool), _i32, _i32, _c_void_p, _c_void_p, _c_void_p,
                                      _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _i32, _c_void_p, _c_void_p]),
    "g4_kv4_gather": (_i32, [_P(G4LayerParams), _P(G4KV4Pool), _i32, _i32, _c_void_p, _i32, _c_void_p, _c_void_p,
                             _i32, _i32, _c_void_p, _c_void_p, _c_void_p]),
    "g4_kv4_decode_workspace_size": (ctypes.c_size_t, [_P(G4LayerParams), _i32, _i32]),
    "g4_kv4_attn_decode": (_i32, [_P(G4LayerParams), _P(G4KV4Pool), _i32, _i32, _c_void_p, _c_void_p, _i32, _c_void_p,
                                  _i32, _i32, _c_void_p, _c_void_p, ctypes.c_size_t, _c_void_p]),
    "g4_kv4_prefill_workspace_size": (ctypes.c_size_t, [_P(G4LayerParams), _i32, _i32, _i32]),
    "g4_kv4_attn_prefill": (_i32, [_P(G4LayerParams), _P(G4KV4Pool), _i32, _i32, _c_void_p, _c_void_p, _i32,
                                   _c_void_p, _c_void_p, _i32, _i32, _i32, _c_void_p, _c_void_p, ctypes.c_size_t,
                                   _c_void_p]),
    "g4_attn_visible_ranges": (_i32, [_i32] + [_c_void_p] * 4 + [_i32] * 3 + [_c_void_p] * 3),
    "g4_kv_append_normrope_axes": (_i32, [_P(G4LayerParams), _P(G4KVCache), _i32, _i32, _P(G4RopeAxes)] + [_c_void_p] * 7
                                   + [_i32, _i32, _c_void_p, _c_void_p]),
    "g4_attn_prefill_mods": (_i32, [_P(G4LayerParams), _P(G4KVCache), _i32, _i32, _P(G4ScoreMods), _c_void_p, _c_void_p,
                                    _i32, _i32, _c_void_p, _c_void_p]),
    "g4_attn_decode_mods_workspace_size": (ctypes.c_size_t, [_P(G4LayerParams), _i32, _i32]),
    "g4_attn_decode_mods": (_i32, [_P(G4LayerParams), _P(G4KVCache), _i32, _i32, _P(G4ScoreMods), _c_void_p, _c_void_p,
                                   _i32, _i32, _c_void_p, _c_void_p, ctypes.c_size_t, _c_void_p]),
    "g4_last_error": (ctypes.c_char_p, []),
    "g4_take_device_error": (_i32, []),
}

_lib = None


class G4Error(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with python -m gemma_dual_geometry_gb300.build")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(x):
    try:
        return x.data_ptr()
    except AttributeError:
        if x is None or isinstance(x, int):  # an address
            return x
        raise


_raw_stream = None      # device index -> the address of its current stream
_current_device = None  # () -> the current device's index; None where there is one device only


def _find_device_calls():
    global _raw_stream, _current_device
    import torch
    # (building a torch.cuda.Stream object takes as long as a launch)
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if torch.cuda.device_count() > 1:
        _current_device = torch.cuda.current_device
    _raw_stream = get if get is not None else lambda device: torch.cuda.current_stream(device).cuda_stream


def current_stream(device):
    """The address of the current stream of the device with this index."""
    if _raw_stream is None:
        _find_device_calls()
    return _raw_stream(device)


def _stream(stream, *tensors):
    raw = None
    if stream is not None:
        raw = stream if isinstance(stream, int) else stream.cuda_stream
        if raw != 0:
            return raw
    for t in tensors:
        if t is not None and not isinstance(t, int) and t.is_cuda:
            device = t.get_device()
            here = current_stream(device)
            # 0 is every device's default stream, and a launch there goes to the current device
            if _current_device is not None and device != _current_device():
                raise ValueError(f"tensors of cuda:{device}, but the current device is cuda:{_current_device()}: "
                                 f"call under torch.cuda.device({device})")
            return here if raw is None else raw
    return raw


def _check(status):
    if status != G4_OK:
        raise G4Error(status, lib().g4_last_error().decode())


def layer_params(layer_type, head_dim, n_heads, n_kv_heads, window=0, theta=1e4, rotary_fraction=1.0, eps=1e-6,
                 attn_scale=1.0, kv_share_src=-1, dtype=G4_BF16):
    return G4LayerParams(int(layer_type), int(head_dim), int(n_heads), int(n_kv_heads), int(window), float(theta),
                         float(rotary_fraction), float(eps), float(attn_scale), int(kv_share_src), int(dtype))


def cache_table(n_layers):
    """Zeroed array of n_layers g4_kv_cache entries."""
    return (G4KVCache * n_layers)()


def set_cache(table, layer, k, v, layer_type, head_dim, n_kv_heads, max_len, batch, dtype, ring=False):
    """Fill entry ``layer``; ``ring`` makes it a sliding-window ring of max_len rows."""
    table[layer] = G4KVCache(_ptr(k), _ptr(v), int(layer_type), int(head_dim), int(n_kv_heads), int(max_len),
                             int(batch), int(dtype), int(bool(ring)))


def g4_kv_share_src(n_layers, n_shared, is_sliding, layer):
    arr = (ctypes.c_int32 * n_layers)(*[1 if s else 0 for s in is_sliding])
    return lib().g4_kv_share_src(n_layers, n_shared, arr, layer)


def g4_kv_append_normrope(params, caches, layer, q_in, k_in, v_in, q_norm_w, k_norm_w, positions, B, T, q_out,
                          stream=None):
    _check(lib().g4_kv_append_normrope(ctypes.byref(params), caches, len(caches), layer, _ptr(q_in), _ptr(k_in),
                                       _ptr(v_in), _ptr(q_norm_w), _ptr(k_norm_w), _ptr(positions), B, T,
                                       _ptr(q_out), _stream(stream, q_in)))


def g4_attn_prefill(params, caches, layer, q, q_start_pos, B, T, out, stream=None):
    _check(lib().g4_attn_prefill(ctypes.byref(params), caches, len(caches), layer, _ptr(q), _ptr(q_start_pos), B, T,
                                 _ptr(out), _stream(stream, q)))


def g4_attn_encoder(params, caches, layer, q, B, T, out, stream=None):
    _check(lib().g4_attn_encoder(ctypes.byref(params), caches, len(caches), layer, _ptr(q), B, T, _ptr(out),
                                 _stream(stream, q)))


def g4_attn_decode_workspace_size(params, B, max_seq_len):
    return int(lib().g4_attn_decode_workspace_size(ctypes.byref(params), B, max_seq_len))


def g4_attn_decode(params, caches, layer, q, seq_lens, B, max_seq_len, out, workspace=None, workspace_bytes=0,
                   stream=None):
    _check(lib().g4_attn_decode(ctypes.byref(params), caches, len(caches), layer, _ptr(q), _ptr(seq_lens), B,
                                max_seq_len, _ptr(out), _ptr(workspace), int(workspace_bytes), _stream(stream, q)))


def g4_decode_step(params, caches, layer, q_in, k_in, v_in, q_norm_w, k_norm_w, seq_lens, B, max_seq_len, out,
                   workspace=None, workspace_bytes=0, stream=None):
    _check(lib().g4_decode_step(ctypes.byref(params), caches, len(caches), layer, _ptr(q_in), _ptr(k_in), _ptr(v_in),
                                _ptr(q_norm_w), _ptr(k_norm_w), _ptr(seq_lens), B, max_seq_len, _ptr(out),
                                _ptr(workspace), int(workspace_bytes), _stream(stream, q_in)))


G4_NOALLOC_SCRATCH_BYTES = 8 << 20


def g4_attn_decode_noalloc(params, caches, layer, q, seq_lens, B, max_seq_len, out, stream=None):
    """g4_attn_decode with the library's built-in scratch instead of a workspace."""
    _check(lib().g4_attn_decode_noalloc(ctypes.byref(params), caches, len(caches), layer, _ptr(q), _ptr(seq_lens),
                                        B, max_seq_len, _ptr(out), _stream(stream, q)))


def g4_qkv_project_append(params, caches, layer, x, D, w_qkv, q_norm_w, k_norm_w, positions, B, T, q_out,
                          stream=None):
    """q/k/v projections of x (attention-norm weight folded into w_qkv) fused into the norm/RoPE/append."""
    _check(lib().g4_qkv_project_append(ctypes.byref(params), caches, len(caches), layer, _ptr(x), int(D),
                                       _ptr(w_qkv), _ptr(q_norm_w), _ptr(k_norm_w), _ptr(positions), B, T,
                                       _ptr(q_out), _stream(stream, x)))


def g4_attn_out_residual(ao, M, K, w_o, D, post_norm_w, eps, h, out, stream=None):
    """out = h + rmsnorm(ao . w_o^T, post_norm_w, eps)."""
    _check(lib().g4_attn_out_residual(_ptr(ao), int(M), int(K), _ptr(w_o), int(D), _ptr(post_norm_w), float(eps),
                                      _ptr(h), _ptr(out), _stream(stream, ao)))


def kv4_pool_table(n_layers):
    """Zeroed array of n_layers g4_kv4_pool entries."""
    return (G4KV4Pool * n_layers)()


def kv4_pool_bytes(n_blocks, n_kv_heads, block_size, head_dim):
    """Bytes of one layer's pool."""
    return n_blocks * n_kv_heads * (block_size // 16) * 18 * head_dim


def set_kv4_pool(table, layer, data, layer_type, head_dim, n_kv_heads, n_blocks, block_size, k_exp=0):
    """Fill entry ``layer`` of a pool table."""
    table[layer] = G4KV4Pool(_ptr(data), int(layer_type), int(head_dim), int(n_kv_heads), int(n_blocks),
                             int(block_size), int(k_exp))


def g4_kv4_assign_blocks(B, T, block_size, n_blocks, max_blocks, old_lens, new_lens, free_blocks, free_count,
                         block_table, lens_out, free_count_out, positions, slots, stream=None):
    _check(lib().g4_kv4_assign_blocks(B, T, block_size, n_blocks, max_blocks, _ptr(old_lens), _ptr(new_lens),
                                      _ptr(free_blocks), _ptr(free_count), _ptr(block_table), _ptr(lens_out),
                                      _ptr(free_count_out), _ptr(positions), _ptr(slots), _stream(stream, old_lens)))


def g4_kv4_append_normrope(params, pools, layer, q_in, k_in, v_in, q_norm_w, k_norm_w, positions, slots, B, T, q_out,
                           stream=None):
    """g4_kv_append_normrope into a 4-bit pool at the tokens' slots."""
    _check(lib().g4_kv4_append_normrope(ctypes.byref(params), pools, len(pools), layer, _ptr(q_in), _ptr(k_in),
                                        _ptr(v_in), _ptr(q_norm_w), _ptr(k_norm_w), _ptr(positions), _ptr(slots), B,
                                        T, _ptr(q_out), _stream(stream, q_in)))


def g4_kv4_gather(params, pools, layer, block_table, max_blocks, start, seq_lens, B, rows, k_out, v_out, stream=None):
    """Positions [start, start + rows) of every sequence as bf16 rows."""
    _check(lib().g4_kv4_gather(ctypes.byref(params), pools, len(pools), layer, _ptr(block_table), max_blocks,
                               _ptr(start), _ptr(seq_lens), B, rows, _ptr(k_out), _ptr(v_out),
                               _stream(stream, k_out)))


def g4_kv4_decode_workspace_size(params, B, max_seq_len):
    return int(lib().g4_kv4_decode_workspace_size(ctypes.byref(params), B, max_seq_len))


def g4_kv4_attn_decode(params, pools, layer, q, block_table, max_blocks, seq_lens, B, max_seq_len, out,
                       workspace=None, workspace_bytes=0, stream=None):
    _check(lib().g4_kv4_attn_decode(ctypes.byref(params), pools, len(pools), layer, _ptr(q), _ptr(block_table),
                                    max_blocks, _ptr(seq_lens), B, max_seq_len, _ptr(out), _ptr(workspace),
                                    int(workspace_bytes), _stream(stream, q)))


def g4_kv4_prefill_workspace_size(params, B, T, max_seq_len):
    return int(lib().g4_kv4_prefill_workspace_size(ctypes.byref(params), B, T, max_seq_len))


def g4_kv4_attn_prefill(params, pools, layer, q, block_table, max_blocks, q_start_pos, seq_lens, B, T, max_seq_len,
                        out, workspace, workspace_bytes, stream=None):
    _check(lib().g4_kv4_attn_prefill(ctypes.byref(params), pools, len(pools), layer, _ptr(q), _ptr(block_table),
                                     max_blocks, _ptr(q_start_pos), _ptr(seq_lens), B, T, max_seq_len, _ptr(out),
                                     _ptr(workspace), int(workspace_bytes), _stream(stream, q)))


_ANY = 1 << 62  # entries of an array that is given by its address, or not at all


def score_mods(softcap=0.0, slopes=None, key_begin=None, key_end=None):
    """What is done to a layer's scores (g4_score_mods).  Holds on to the tensors that it is made of, which the calls
    refuse where they are on another device than q or have fewer entries than heads or tokens."""
    device, entries = None, []
    for t, dtype in ((slopes, "float32"), (key_begin, "int32"), (key_end, "int32")):
        if t is None or isinstance(t, int):
            entries.append(_ANY)
            continue
        if str(t.dtype) != "torch." + dtype or not t.is_contiguous():
            raise ValueError(f"expected a contiguous tensor of {dtype}, got one of {t.dtype}")
        if device is not None and t.get_device() != device:
            raise ValueError("slopes, key_begin and key_end are on different devices")
        device = t.get_device()
        entries.append(t.numel())
    m = G4ScoreMods(float(softcap), _ptr(slopes), _ptr(key_begin), _ptr(key_end))
    m.tensors = (slopes, key_begin, key_end)
    m.device, m.entries = device, entries
    return m


def rope_axes(n_axes, axis, head_dim, inv_freq=None):
    """Positions of several axes (g4_rope_axes): ``axis[j]`` turns pair j, ``inv_freq[j]`` is its frequency (None: the
    layer's).  Both may stop at the layer's last rotated pair, no earlier (the call refuses that)."""
    half = head_dim // 2
    for given in (axis, inv_freq):
        if given is not None and len(given) > half:
            raise ValueError(f"{len(given)} pairs in a head of {half}")
    if not all(0 <= x < 256 and x == int(x) for x in axis):  # (an 8-bit table would take them modulo 256)
        raise ValueError("axes are whole numbers from 0 on")
    table = (ctypes.c_uint8 * half)(*[int(x) for x in axis])
    freq = None if inv_freq is None else (ctypes.c_float * half)(*[float(x) for x in inv_freq])
    axes = G4RopeAxes(int(n_axes), ctypes.cast(table, _P(ctypes.c_uint8)),
                      None if freq is None else ctypes.cast(freq, _P(ctypes.c_float)))
    axes.pairs = len(axis) if inv_freq is None else min(len(axis), len(inv_freq))
    return axes


def g4_attn_visible_ranges(window, q_start_pos, seq_lens, doc_ids, span_ids, max_len, B, T, key_begin, key_end,
                           stream=None):
    """The interval of keys that each token sees, from documents and spans."""
    _check(lib().g4_attn_visible_ranges(window, _ptr(q_start_pos), _ptr(seq_lens), _ptr(doc_ids), _ptr(span_ids),
                                        max_len, B, T, _ptr(key_begin), _ptr(key_end), _stream(stream, q_start_pos)))


def g4_kv_append_normrope_axes(params, caches, layer, axes, q_in, k_in, v_in, q_norm_w, k_norm_w, positions, rows, B, T,
                               q_out, stream=None):
    """g4_kv_append_normrope with positions of several axes [n_axes][B][T], apart from the cache's rows [B][T]."""
    pairs = getattr(axes, "pairs", _ANY)  # (a structure of the caller's own)
    if pairs < params.head_dim // 2:
        turned = int(params.head_dim * params.rotary_fraction / 2)
        if pairs < turned:
            raise ValueError(f"axes or frequencies of {pairs} pairs, but the layer turns {turned}")
    _check(lib().g4_kv_append_normrope_axes(ctypes.byref(params), caches, len(caches), layer, ctypes.byref(axes),
                                            _ptr(q_in), _ptr(k_in), _ptr(v_in), _ptr(q_norm_w), _ptr(k_norm_w),
                                            _ptr(positions), _ptr(rows), B, T, _ptr(q_out), _stream(stream, q_in)))


def _mods(mods, q, heads, tokens):
    """The address of a call's mods, whose tensors the kernels can read: of q's device, an entry for every head or token."""
    if mods is None:
        return None
    device = getattr(mods, "device", None)  # (None: no tensors, or a structure of the caller's own)
    if device is not None:
        if device < 0 or (q is not None and not isinstance(q, int) and q.get_device() != device):
            raise ValueError("slopes, key_begin and key_end must be on the device of q")
        slopes, begin, end = mods.entries
        if slopes < heads or begin < tokens or end < tokens:
            raise ValueError(f"slopes need {heads} entries, key_begin and key_end {tokens}")
    return ctypes.byref(mods)


def g4_attn_prefill_mods(params, caches, layer, mods, q, q_start_pos, B, T, out, stream=None):
    """g4_attn_prefill with modified scores (score_mods(), or None)."""
    _check(lib().g4_attn_prefill_mods(ctypes.byref(params), caches, len(caches), layer,
                                      _mods(mods, q, params.n_heads, B * T), _ptr(q), _ptr(q_start_pos), B, T,
                                      _ptr(out), _stream(stream, q)))


def g4_attn_decode_mods_workspace_size(params, B, max_seq_len):
    return int(lib().g4_attn_decode_mods_workspace_size(ctypes.byref(params), B, max_seq_len))


def g4_attn_decode_mods(params, caches, layer, mods, q, seq_lens, B, max_seq_len, out, workspace=None,
                        workspace_bytes=0, stream=None):
    """g4_attn_decode with modified scores (score_mods(), or None)."""
    _check(lib().g4_attn_decode_mods(ctypes.byref(params), caches, len(caches), layer,
                                     _mods(mods, q, params.n_heads, B), _ptr(q), _ptr(seq_lens), B, max_seq_len,
                                     _ptr(out), _ptr(workspace), int(workspace_bytes), _stream(stream, q)))


def g4_last_error():
    return lib().g4_last_error().decode()


def g4_take_device_error():
    return int(lib().g4_take_device_error())
