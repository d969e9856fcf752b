"""Host-side driver of an attention-only layer stack over the C ABI.

Owns the device buffers of a stack (one KV cache per layer that owns one,
q_out scratch per head width, decode workspaces) and sequences the per-layer
calls: g4_kv_append_normrope then g4_attn_prefill / g4_attn_decode (or
g4_attn_encoder), with modified scores and positions of several axes where asked.
Sliding caches may be rings of one window.  Shared-KV
tail layers get no cache and read their source layer's
(cortiq-engine g4e.rs `g4e_forward`: `src = kv_share_src.unwrap_or(li)`).
``PagedAttnStack`` is the same over the paged 4-bit cache: g4_kv4_assign_blocks
once per step for all layers, then per layer g4_kv4_append_normrope and
g4_kv4_attn_prefill / g4_kv4_attn_decode.
Every step runs in the CUDA kernels; this module only allocates and calls.
"""

from __future__ import annotations

import contextlib

import torch

from . import g4attn as G
from . import workloads as W


def _layers(cfg):
    """Source layer, geometry and parameters of every layer."""
    n = len(cfg["types"])
    is_s = [t == W.SLIDING for t in cfg["types"]]
    src = [G.g4_kv_share_src(n, cfg["n_shared"], is_s, l) for l in range(n)]
    if any(s == -2 for s in src):
        raise ValueError("invalid shared-KV routing for this stack")
    geo = [W.layer_geometry(cfg, l) for l in range(n)]
    params = [G.layer_params(g["layer_type"], g["head_dim"], g["n_heads"], g["n_kv_heads"], g["window"],
                             g["theta"], g["rotary_fraction"], g["eps"], g["attn_scale"], src[l],
                             g["dtype"]) for l, g in enumerate(geo)]
    return src, geo, params


class AttnStack:
    def __init__(self, cfg, Lmax, device="cuda", B=None, mods=False):
        """``mods``: there will be decodes with modified scores (one more workspace per layer)."""
        self.cfg = cfg
        self.B = cfg["B"] if B is None else B
        self.Lmax = Lmax
        self.device = torch.device(device)
        self.n = len(cfg["types"])
        self.src, self.geo, self.params = _layers(cfg)
        self.table = G.cache_table(self.n)
        self.caches = {}
        tdt = W.torch_dtype(cfg["dtype"])
        for l, g in enumerate(self.geo):
            if self.src[l] < 0:
                # a ring (sliding layers of a ring workload) holds one window
                rows = W.cache_rows(cfg, l, Lmax)
                shape = (self.B, cfg["Hkv"], rows, g["head_dim"])
                k = torch.zeros(shape, dtype=tdt, device=self.device)
                v = torch.zeros(shape, dtype=tdt, device=self.device)
                self.caches[l] = (k, v)
                G.set_cache(self.table, l, k, v, g["layer_type"], g["head_dim"], cfg["Hkv"], rows, self.B,
                            cfg["dtype"], ring=bool(cfg.get("ring")) and g["layer_type"] == W.SLIDING)
        self.ws = {}
        for l, p in enumerate(self.params):
            nb = G.g4_attn_decode_workspace_size(p, self.B, Lmax)
            self.ws[l] = (torch.zeros(max(nb, 16), dtype=torch.uint8, device=self.device), nb)
        self.mods_ws = {}
        if mods:
            for l, p in enumerate(self.params):
                nb = G.g4_attn_decode_mods_workspace_size(p, self.B, Lmax)
                self.mods_ws[l] = torch.zeros(max(nb, 16), dtype=torch.uint8, device=self.device)
        if self.device.type == "cuda":
            torch.cuda.current_stream(self.device).synchronize()  # what was queued above is there for any stream

    def owns(self, l):
        return self.src[l] < 0

    def cache_bytes(self):
        return sum(k.numel() * k.element_size() * 2 for k, _ in self.caches.values())

    def visible_ranges(self, layer_type, q_start, seq_lens, doc_ids, span_ids, T, key_begin, key_end, stream=None):
        """The intervals of keys of T tokens per sequence, for all layers of one type (ids are [B][Lmax])."""
        windows = [g["window"] for g in self.geo if g["layer_type"] == layer_type]
        if not windows:
            raise ValueError(f"the stack has no layers of type {layer_type}")
        for what, x, n in (("q_start", q_start, 1), ("seq_lens", seq_lens, 1), ("doc_ids", doc_ids, self.Lmax),
                           ("span_ids", span_ids, self.Lmax), ("key_begin", key_begin, T), ("key_end", key_end, T)):
            self._check_i32(what, x, self.B * n)
        G.g4_attn_visible_ranges(windows[0] if layer_type == W.SLIDING else 0, q_start, seq_lens, doc_ids, span_ids,
                                 self.Lmax, self.B, T, key_begin, key_end, stream=stream)

    def append_axes(self, l, axes, q, k, v, qw, kw, positions, rows, T, q_out, stream=None):
        """append() with positions of several axes [n_axes][B][T], apart from the cache's rows [B][T]."""
        rows = rows if self.owns(l) else None
        self._check_i32("positions", positions, axes.n_axes * self.B * T)
        self._check_i32("rows", rows, self.B * T)
        G.g4_kv_append_normrope_axes(self.params[l], self.table, l, axes, q, k, v, qw, kw, positions, rows, self.B, T,
                                     q_out, stream=stream)

    @staticmethod
    def _check_i32(what, x, n):
        """Whether tensor ``x`` (not an address, nor None) is what the kernels read n 32-bit numbers of."""
        if x is None or isinstance(x, int):
            return
        few = x.numel() < n if x.dim() == 1 else x.numel() != n   # (a flat buffer may be longer)
        if x.dtype != torch.int32 or few or not x.is_contiguous():
            raise ValueError(f"{what} must be {n} int32 numbers, contiguous")

    def append(self, l, q, k, v, qw, kw, positions, T, q_out, stream=None):
        G.g4_kv_append_normrope(self.params[l], self.table, l, q, k, v, qw, kw, positions, self.B, T, q_out,
                                stream=stream)

    def prefill_attn(self, l, q_out, q_start, T, out, stream=None, mods=None):
        """``mods``: G.score_mods(), for modified scores."""
        if mods is not None:
            G.g4_attn_prefill_mods(self.params[l], self.table, l, mods, q_out, q_start, self.B, T, out, stream=stream)
            return
        G.g4_attn_prefill(self.params[l], self.table, l, q_out, q_start, self.B, T, out, stream=stream)

    def encoder_attn(self, l, q_out, T, out, stream=None):
        """Bidirectional attention over the T tokens appended at positions 0..T-1."""
        G.g4_attn_encoder(self.params[l], self.table, l, q_out, self.B, T, out, stream=stream)

    def decode_attn(self, l, q_out, seq_lens, max_seq_len, out, stream=None, mods=None):
        if mods is not None:
            if not self.mods_ws:
                raise ValueError("the stack was made without mods")
            ws = self.mods_ws[l]
            G.g4_attn_decode_mods(self.params[l], self.table, l, mods, q_out, seq_lens, self.B, max_seq_len, out,
                                  ws, ws.numel(), stream=stream)
            return
        ws, nb = self.ws[l]
        G.g4_attn_decode(self.params[l], self.table, l, q_out, seq_lens, self.B, max_seq_len, out, ws, nb,
                         stream=stream)

    def decode_step(self, l, q, k, v, qw, kw, seq_lens, max_seq_len, out, stream=None):
        """Fused append of the new token + decode attention (one launch)."""
        ws, nb = self.ws[l]
        G.g4_decode_step(self.params[l], self.table, l, q, k, v, qw, kw, seq_lens, self.B, max_seq_len, out, ws, nb,
                         stream=stream)

    def decode_launches(self, l):
        """Kernels one g4_attn_decode or g4_decode_step call launches."""
        return 1


class PagedAttnStack:
    """A stack over the paged 4-bit cache: B sequence slots of at most max_len positions, whose layers share
    one block table and n_blocks blocks of block_size positions.  ``k_exp`` as in g4_kv4_pool.

    Calls may go to any stream, one after another.  The stack's memory stays its own until the streams that it was
    used on (torch's; not addresses) are done with it, also when the stack goes before that."""

    def __init__(self, cfg, max_len, n_blocks, block_size=64, device="cuda", B=None, k_exp=0):
        self.cfg = cfg
        self.B = cfg["B"] if B is None else B
        self.device = torch.device(device)
        self.n = len(cfg["types"])
        self.n_blocks, self.block_size = n_blocks, block_size
        self.max_blocks = -(-max_len // block_size)
        self.max_len = self.max_blocks * block_size
        self.src, self.geo, self.params = _layers(cfg)
        self.table = G.kv4_pool_table(self.n)
        self.pools = {}
        for l, g in enumerate(self.geo):
            if self.src[l] < 0:
                size = G.kv4_pool_bytes(n_blocks, cfg["Hkv"], block_size, g["head_dim"])
                self.pools[l] = torch.zeros(size, dtype=torch.uint8, device=self.device)
                G.set_kv4_pool(self.table, l, self.pools[l], g["layer_type"], g["head_dim"], cfg["Hkv"], n_blocks,
                               block_size, k_exp)

        def i32(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=self.device)

        self.block_table = i32(self.B, self.max_blocks)
        self.free_blocks = torch.arange(n_blocks, dtype=torch.int32, device=self.device)
        self.free_count = torch.full((1,), n_blocks, dtype=torch.int32, device=self.device)
        self.lens = i32(self.B)    # positions held
        self.start = i32(self.B)   # and held before the last assign()
        # one decode workspace serves all layers in turn
        self.ws_bytes = max(G.g4_kv4_decode_workspace_size(p, self.B, self.max_len) for p in self.params)
        self.ws = torch.zeros(max(self.ws_bytes, 16), dtype=torch.uint8, device=self.device)
        self._streams = {}         # address -> stream, of those that have used the buffers
        self._by_address = False   # whether others have, of which the address is all that is known
        if self.device.type == "cuda":
            home = torch.cuda.current_stream(self.device)
            home.synchronize()     # what was queued above is there for any stream
            self._streams[home.cuda_stream] = home
        self._i32 = i32
        self._steps = {}           # T -> (positions, slots)
        self._no_ws = torch.empty(0, dtype=torch.uint8, device=self.device)
        self._prefill_ws, self._prefill_T = self._no_ws, 0  # one workspace for prefills of up to so many tokens
        self._captured_ws = False  # whether a graph was captured with it
        self._kept_ws = []         # outgrown ones that graphs still use

    def _buffers(self):
        own = [self.block_table, self.free_blocks, self.free_count, self.lens, self.start, self.ws, self._prefill_ws]
        return own + [*self.pools.values(), *self._kept_ws, *(t for step in self._steps.values() for t in step)]

    def _use(self, stream):
        """A call is about to go to ``stream``: no buffer is anyone else's before that stream is done with it."""
        if isinstance(stream, int):
            self._by_address = True
            return
        if self.device.type != "cuda":
            return
        at = G.current_stream(self.lens.get_device()) if stream is None else stream.cuda_stream
        if at not in self._streams:
            self._streams[at] = torch.cuda.current_stream(self.device) if stream is None else stream
            for t in self._buffers():
                t.record_stream(self._streams[at])

    def _new(self, t):
        """A buffer taken later may come to be used on all those streams."""
        for s in self._streams.values():
            t.record_stream(s)
        return t

    def _step(self, T):
        if T not in self._steps:
            self._steps[T] = self._new(self._i32(self.B, T)), self._new(self._i32(self.B, T))
        return self._steps[T]

    def _wait_for_all(self):
        if self.device.type == "cuda":
            torch.cuda.synchronize(self.device)

    def _capturing(self, stream):
        if self.device.type != "cuda":
            return False
        with self._on(stream):
            return torch.cuda.is_current_stream_capturing()

    def _prefill_workspace(self, T, stream):
        """The workspace of the longest prefill yet, which serves all of them in turn; outgrown ones go, but for
        those that a graph was captured with."""
        if self._prefill_T < T <= self.max_len:   # (more are the call's to refuse)
            size = max(G.g4_kv4_prefill_workspace_size(p, self.B, T, self.max_len) for p in self.params)
            if self._captured_ws or (self._by_address and self._capturing(stream)):
                self._kept_ws.append(self._prefill_ws)
            elif self._by_address and self._prefill_T > 0:
                self._wait_for_all()
            self._prefill_ws, self._prefill_T, self._captured_ws = self._no_ws, 0, False  # (gone before the next is taken)
            with self._on(stream):
                self._prefill_ws = self._new(torch.empty(size, dtype=torch.uint8, device=self.device))
            self._prefill_T = T
        self._captured_ws = self._captured_ws or self._capturing(stream)
        return self._prefill_ws

    def _on(self, stream):
        """What torch does within runs on ``stream`` (a stream, an address, or None: the current one)."""
        if stream is None:
            return contextlib.nullcontext()
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.device)
        return torch.cuda.stream(stream)

    def owns(self, l):
        return self.src[l] < 0

    def cache_bytes(self):
        return sum(p.numel() for p in self.pools.values())

    def assign(self, new_lens, T, stream=None):
        """Blocks for sequences that go to new_lens [B] (int32) positions with T new tokens at most (0 ends one).
        Sets ``lens`` (what was granted) and ``start``; the T tokens' positions and slots serve append()."""
        if not isinstance(new_lens, int):   # (an address)
            like = self.lens
            if not (isinstance(new_lens, torch.Tensor) and new_lens.dtype == like.dtype and new_lens.numel() == self.B
                    and new_lens.get_device() == like.get_device() and new_lens.is_contiguous()):
                raise ValueError(f"new_lens must be {self.B} int32 lengths, contiguous, on the stack's device")
        self._use(stream)
        with self._on(stream):
            positions, slots = self._step(T)
            self.start.copy_(self.lens)
        G.g4_kv4_assign_blocks(self.B, T, self.block_size, self.n_blocks, self.max_blocks, self.lens, new_lens,
                               self.free_blocks, self.free_count, self.block_table, self.lens, self.free_count,
                               positions, slots, stream=stream)
        return positions, slots

    def append(self, l, q, k, v, qw, kw, T, q_out, stream=None):
        if T not in self._steps:
            raise ValueError(f"append of {T} tokens per sequence: assign() gave out no slots for so many")
        self._use(stream)
        positions, slots = self._step(T)
        G.g4_kv4_append_normrope(self.params[l], self.table, l, q, k, v, qw, kw, positions,
                                 slots if self.owns(l) else None, self.B, T, q_out, stream=stream)

    def prefill_attn(self, l, q_out, T, out, stream=None):
        self._use(stream)
        ws = self._prefill_workspace(T, stream)
        G.g4_kv4_attn_prefill(self.params[l], self.table, l, q_out, self.block_table, self.max_blocks, self.start,
                              self.lens, self.B, T, self.max_len, out, ws, ws.numel(), stream=stream)

    def decode_attn(self, l, q_out, out, stream=None):
        self._use(stream)
        G.g4_kv4_attn_decode(self.params[l], self.table, l, q_out, self.block_table, self.max_blocks, self.lens,
                             self.B, self.max_len, out, self.ws, self.ws_bytes, stream=stream)

    def gather(self, l, start, rows, k_out, v_out, stream=None):
        """Positions [start[b], start[b] + rows) of every sequence as bf16 rows."""
        self._use(stream)
        G.g4_kv4_gather(self.params[l], self.table, l, self.block_table, self.max_blocks, start, self.lens, self.B,
                        rows, k_out, v_out, stream=stream)
