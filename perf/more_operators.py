"""Cases that measure attention with modified scores and what feeds it.

Four operators, for prompts with images, packed documents and capped scores:

  ranges   the interval of keys that each token sees, from the documents that a
           row of tokens is packed of and the spans (images, prefixes) within
           which tokens see each other in both directions;
  append   norm and RoPE of q and k with several position axes (time, height,
           width), norm of v, k and v written to the cache's rows;
  prefill  attention of new tokens whose scores are capped by a tanh, get a
           bias that falls with distance, and reach an interval of keys each;
  decode   the same for one new token per sequence.

``run`` computes them in plain torch operations where ``own`` is false and
calls the library where it is true.  Caches are [B][Hkv][rows][hd]; position p
lies in row p, or in row p mod rows where the cache is a ring.
"""

import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
EPS = 1e-6
# theta and the rotated part of a head on sliding and on full layers
THETA = {True: 1e4, False: 1e6}
ROTATED = {True: 1.0, False: 0.25}
AXES = 3


# ------------------------------------------------------------------ the cases

def listed():
    full = dict(H=8, Hkv=2, hd=512, window=0, ring=False, dtype="bf16")
    slide = dict(H=8, Hkv=2, hd=256, window=512, ring=False, dtype="bf16")
    return [
        # one prompt of a few documents and images on a sliding layer, where latency counts
        dict(name="ranges 1x1000", op="ranges", B=1, T=1000, lo=0, hi=0, window=512, doc=300, span=100),
        # rows of 32768 positions packed of documents with images, on a full layer
        dict(name="ranges 8x32768", op="ranges", B=8, T=32768, lo=0, hi=0, window=0, doc=2000, span=256),
        # the new token of 64 sequences into rings of one window
        dict(name="append step 64 sliding ring", op="append", B=64, T=1, lo=1024, hi=8192, span=0, mixed=False,
             **dict(slide, ring=True)),
        # a prompt chunk of 8 sequences with images on a full layer
        dict(name="append 8x2048 full", op="append", B=8, T=2048, lo=0, hi=2048, span=256, mixed=False, **full),
        # a few odd tokens in float32, axes that take turns
        dict(name="append 3x101 f32", op="append", B=3, T=101, lo=0, hi=50, span=40, mixed=True, H=4, Hkv=2, hd=128,
             window=0, ring=False, dtype="f32"),
        # the smallest prefill: a short prompt with capped scores
        dict(name="prefill 1x77 capped", op="prefill", B=1, T=77, lo=0, hi=0, mask="causal", cap=50.0, bias=False, H=4,
             Hkv=2, hd=64, window=0, ring=False, dtype="bf16"),
        # a row of 8192 tokens packed of documents with images, on a sliding layer
        dict(name="prefill 1x8192 packed sliding", op="prefill", B=1, T=8192, lo=0, hi=0, mask="both", doc=1000, span=200,
             cap=0.0, bias=False, **slide),
        # prompts of 4 sequences with images on a full layer, capped
        dict(name="prefill 4x2048 images full capped", op="prefill", B=4, T=2048, lo=0, hi=500, mask="spans", span=256,
             cap=50.0, bias=False, **full),
        # two long prompts with a distance bias
        dict(name="prefill 2x4096 bias", op="prefill", B=2, T=4096, lo=0, hi=0, mask="causal", cap=0.0, bias=True,
             **dict(full, hd=128)),
        # the smallest decode: one short sequence, capped
        dict(name="decode 1x333 capped", op="decode", B=1, lo=333, hi=333, cap=50.0, bias=False, begin=False, H=8, Hkv=1,
             hd=128, window=0, ring=False, dtype="bf16"),
        # a serving batch on a full layer, capped
        dict(name="decode 64 full capped", op="decode", B=64, lo=1024, hi=8192, cap=50.0, bias=False, begin=False, **full),
        # few sequences of a long context: distance bias, sequences that begin behind padding
        dict(name="decode 4x131072 full bias", op="decode", B=4, lo=131072, hi=131072, cap=0.0, bias=True, begin=True,
             **full),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is spread evenly over lo .. hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ranges", "append", "prefill", "prefill", "prefill", "decode", "decode"])
    if op == "ranges":
        T, hi = _log(rng, 1, 16384), rng.choice([0, _log(rng, 1, 60000)])
        return dict(op=op, B=_log(rng, 1, max(1, (1 << 18) // (T + hi))), T=T, lo=rng.randrange(0, hi + 1), hi=hi,
                    window=rng.choice([0, _log(rng, 1, 2000)]), doc=rng.choice([0, _log(rng, 2, 5000)]),
                    span=rng.choice([0, _log(rng, 1, 1000)]))
    hd = rng.choice([64, 128, 256, 512])
    group = rng.choice([g for g in (1, 2, 4, 8) if g * hd <= 2048])
    Hkv = rng.choice([1, 2, 2, 3])
    window = rng.choice([0, _log(rng, 1, 1500)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    c = dict(op=op, H=group * Hkv, Hkv=Hkv, hd=hd, window=window, ring=False, dtype=dtype)
    scores = dict(cap=rng.choice([0.0, 50.0, 30.0, round(rng.uniform(2.0, 100.0), 2)]), bias=rng.random() < 0.4)
    # a drawn case stays below the largest listed one
    if op == "append":
        T = rng.choice([1, _log(rng, 2, 2048)])
        most = max(1, (1 << 26) // (T * (c["H"] + 2 * Hkv) * hd))
        hi = _log(rng, 1, 4000)
        c.update(B=_log(rng, 1, min(128, most)), T=T, lo=rng.randrange(0, hi + 1), hi=hi, span=rng.choice([0, _log(rng, 2, 500)]),
                 mixed=rng.random() < 0.5, ring=T == 1 and window > 0 and rng.random() < 0.5)
    elif op == "prefill":
        small = dtype == "f32"  # (float32 attention is for small models)
        T, hi = _log(rng, 1, 300 if small else 3000), rng.choice([0, _log(rng, 1, 300 if small else 4000)])
        most = max(1, (1 << (22 if small else 27)) // (c["H"] * T * (T + hi)))
        mask = rng.choice(["causal", "docs", "spans", "both"])
        c.update(B=_log(rng, 1, min(8, most)), T=T, lo=rng.randrange(0, hi + 1), hi=hi, mask=mask, doc=_log(rng, 2, 2000),
                 span=_log(rng, 1, 500), ring=mask == "causal" and window > 0 and rng.random() < 0.3, **scores)
    else:
        hi = _log(rng, 1, 30000)
        most = max(1, (1 << 27) // (hi * Hkv * hd))
        c.update(B=_log(rng, 1, min(200, most)), lo=rng.randrange(1, hi + 1), hi=hi, begin=rng.random() < 0.4,
                 ring=window > 0 and rng.random() < 0.3, **scores)
    return c


# ------------------------------------------------------------------ the inputs

def _type(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _unit(shape, gen, dtype):
    """Rows of unit mean square, as a cache is appended."""
    x = torch.randn(shape, generator=gen, device=DEVICE)
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)).to(dtype)


def _ints(lo, hi, n, gen):
    return torch.randint(lo, hi + 1, (n,), generator=gen, device=DEVICE, dtype=torch.int32)


def _segments(B, L, mean, gen):
    """Numbers of the segments, about `mean` positions each, that rows of L positions are cut into."""
    return (torch.rand((B, L), generator=gen, device=DEVICE) < 1.0 / mean).cumsum(1).int()


def _spans(B, L, mean, gen):
    """Every other segment is a span (the first one at times, as a prefix); -1 where tokens see what is before them."""
    seg = _segments(B, L, mean, gen)
    first = torch.randint(0, 2, (B, 1), generator=gen, device=DEVICE, dtype=torch.int32)
    return torch.where(seg % 2 == first, seg, -1).int()


def _runs(ids):
    """Where the run of equal neighbours that each position lies in begins and ends."""
    at = torch.arange(ids.shape[1], device=ids.device).expand_as(ids)
    cut = torch.ones_like(ids, dtype=torch.bool)
    cut[:, 1:] = ids[:, 1:] != ids[:, :-1]
    begin = torch.where(cut, at, 0).cummax(1).values
    last = torch.ones_like(cut)
    last[:, :-1] = cut[:, 1:]
    end = torch.where(last, at + 1, ids.shape[1]).flip(1).cummin(1).values.flip(1)
    return begin, end


def _visible(start, lens, doc, span, T, window):
    """The interval of keys of the tokens at positions start[b] + t, of lens[b] positions that the sequence holds; empty
    past lens[b] and where doc is below 0.  Documents and spans are runs of equal neighbours in doc and span, a span ends
    with its document, and span is below 0 outside of spans."""
    L = doc.shape[1]
    held = torch.arange(L, device=doc.device)[None, :] < lens[:, None]
    lowest = torch.iinfo(torch.int64).min
    doc = torch.where(held, doc.long(), lowest)
    doc_begin, _ = _runs(doc)
    both = doc_begin * (1 << 33) + torch.where(held, span.long(), -(1 << 32))  # (a span in two documents is two)
    span_begin, span_end = _runs(both)
    at = start.long()[:, None] + torch.arange(T, device=doc.device)[None, :]
    p = at.clamp(0, L - 1)
    sees = (at >= 0) & (at < lens[:, None]) & (doc.gather(1, p) >= 0)
    begin, end = doc_begin.gather(1, p), at + 1
    if window:
        begin = torch.maximum(begin, at - (window - 1))
    in_span = span.long().gather(1, p) >= 0
    begin = torch.where(in_span, torch.minimum(begin, span_begin.gather(1, p)), begin)
    end = torch.where(in_span, span_end.gather(1, p), end)
    return torch.where(sees, begin, 0).int(), torch.where(sees, end, 0).int()


def _axis(c):
    """The axis that turns each rotated pair: blocks of an eighth and a half more for height and width, or by turns."""
    turns = int(c["hd"] * ROTATED[c["window"] > 0] / 2)
    if c["mixed"]:
        return [j % AXES for j in range(turns)]
    t, h = turns // 4, turns // 4 + turns * 3 // 8
    return [0 if j < t else 1 if j < h else 2 for j in range(turns)]


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    st = dict(case=c)
    B, T, window = c["B"], c.get("T", 1), c["window"]
    if c["op"] == "ranges":
        start = _ints(c["lo"], c["hi"], B, gen)
        fresh = _ints((T + 1) // 2, T, B, gen)
        L = c["hi"] + T
        doc = _segments(B, L, c["doc"], gen) if c["doc"] else torch.zeros((B, L), dtype=torch.int32, device=DEVICE)
        span = _spans(B, L, c["span"], gen) if c["span"] else torch.full((B, L), -1, dtype=torch.int32, device=DEVICE)
        st.update(start=start, lens=start + fresh, doc=doc, span=span)
    elif c["op"] == "append":
        H, Hkv, hd, dtype = c["H"], c["Hkv"], c["hd"], _type(c)
        start = _ints(c["lo"], c["hi"], B, gen)
        fresh = _ints((T + 1) // 2, T, B, gen)
        t = torch.arange(T, device=DEVICE, dtype=torch.int32)[None, :]
        at = start[:, None] + t
        positions = at[None].repeat(AXES, 1, 1)
        if c["span"]:
            # an image's tokens share a time and lie on a grid 16 wide
            span = _spans(B, T, c["span"], gen)
            begin, _ = _runs(span)
            i = (t - begin).int()
            first = (start[:, None] + begin).int()
            image = torch.stack([first, first + i // 16, first + i % 16])
            positions = torch.where(span >= 0, image, positions)
        rows = torch.where(t < fresh[:, None], at, -1).int()
        cache = torch.zeros((B, Hkv, window if c["ring"] else c["hi"] + T + 1, hd), dtype=dtype, device=DEVICE)
        weight = lambda: 1.0 + 0.1 * torch.randn(hd, generator=gen, device=DEVICE)  # noqa: E731
        row = lambda heads: torch.randn((B, T, heads, hd), generator=gen, device=DEVICE).to(dtype)  # noqa: E731
        st.update(q=row(H), k=row(Hkv), v=row(Hkv), qw=weight(), kw=weight(), positions=positions.int().contiguous(),
                  rows=rows, ck=cache, cv=cache.clone())
    else:
        H, Hkv, hd, dtype = c["H"], c["Hkv"], c["hd"], _type(c)
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEVICE) / H) if c["bias"] else None
        if c["op"] == "prefill":
            start = _ints(c["lo"], c["hi"], B, gen)
            # where tokens have intervals of their own, sequences may be padded
            lens = start + (T if c["mask"] == "causal" else _ints((3 * T + 3) // 4, T, B, gen))
            L = c["hi"] + T
            st["begin"] = st["end"] = None
            if c["mask"] != "causal":
                none = torch.zeros((B, L), dtype=torch.int32, device=DEVICE)
                doc = _segments(B, L, c["doc"], gen) if c["mask"] != "spans" else none
                span = _spans(B, L, c["span"], gen) if c["mask"] != "docs" else none - 1
                st["begin"], st["end"] = _visible(start, lens, doc, span, T, window)
            st["start"], st["q"] = start, _unit((B, T, H, hd), gen, dtype)
            rows = -(-(T + window - 1) // 128) * 128 if c["ring"] else L
        else:
            lens = _ints(c["lo"], c["hi"], B, gen)
            st["begin"] = (torch.rand(B, generator=gen, device=DEVICE).square() * (lens + 1)).int() if c["begin"] else None
            st["q"] = _unit((B, H, hd), gen, dtype)
            rows = window if c["ring"] else c["hi"]
        k, v = _unit((B, Hkv, rows, hd), gen, dtype), _unit((B, Hkv, rows, hd), gen, dtype)
        if not c["ring"]:  # rows that no position has been written to hold anything
            empty = (torch.arange(rows, device=DEVICE)[None, :] >= lens[:, None])[:, None, :, None]
            k.masked_fill_(empty, math.nan)
            v.masked_fill_(empty, math.nan)
        st.update(lens=lens, ck=k, cv=v)
    if own:
        st["kept"] = _kept(st)  # handles, workspaces and output buffers that a program keeps; no data is laid out
    return st


# ------------------------------------------------------------------ the library's calls

def _kept(st):
    from gemma_dual_geometry_gb300 import g4attn as G
    c, z = st["case"], {}
    if c["op"] == "ranges":
        z.update(begin=torch.empty((c["B"], c["T"]), dtype=torch.int32, device=DEVICE))
        z.update(end=torch.empty_like(z["begin"]))
        return z
    kind = G.G4_SLIDING if c["window"] else G.G4_FULL
    dtype = G.G4_BF16 if c["dtype"] == "bf16" else G.G4_F32
    z["params"] = p = G.layer_params(kind, c["hd"], c["H"], c["Hkv"], c["window"], THETA[c["window"] > 0],
                                     ROTATED[c["window"] > 0], EPS, 1.0, -1, dtype)
    z["caches"] = G.cache_table(1)
    G.set_cache(z["caches"], 0, st["ck"], st["cv"], kind, c["hd"], c["Hkv"], st["ck"].shape[2], c["B"], dtype, c["ring"])
    z["out"] = torch.empty_like(st["q"])
    if c["op"] == "append":
        z["axes"] = G.rope_axes(AXES, _axis(c), c["hd"])
    elif c["op"] == "prefill":
        z["mods"] = G.score_mods(c["cap"], st["slopes"], st["begin"], st["end"])
    else:
        z["mods"] = G.score_mods(c["cap"], st["slopes"], st["begin"])
        z["bytes"] = G.g4_attn_decode_mods_workspace_size(p, c["B"], c["hi"])
        z["ws"] = torch.zeros(max(16, z["bytes"]), dtype=torch.uint8, device=DEVICE)
    return z


def _run_own(st):
    from gemma_dual_geometry_gb300 import g4attn as G
    c, z = st["case"], st["kept"]
    if c["op"] == "ranges":
        G.g4_attn_visible_ranges(c["window"], st["start"], st["lens"], st["doc"], st["span"], c["hi"] + c["T"], c["B"],
                                 c["T"], z["begin"], z["end"])
        return dict(begin=z["begin"], end=z["end"])
    if c["op"] == "append":
        G.g4_kv_append_normrope_axes(z["params"], z["caches"], 0, z["axes"], st["q"], st["k"], st["v"], st["qw"], st["kw"],
                                     st["positions"], st["rows"], c["B"], c["T"], z["out"])
        return dict(q=z["out"], k=st["ck"], v=st["cv"])
    if c["op"] == "prefill":
        G.g4_attn_prefill_mods(z["params"], z["caches"], 0, z["mods"], st["q"], st["start"], c["B"], c["T"], z["out"])
    else:
        G.g4_attn_decode_mods(z["params"], z["caches"], 0, z["mods"], st["q"], st["lens"], c["B"], c["hi"], z["out"],
                              z["ws"], z["bytes"])
    return z["out"]


# ------------------------------------------------------------------ the plain forms

def _ranges(st):
    c = st["case"]
    begin, end = _visible(st["start"], st["lens"], st["doc"], st["span"], c["T"], c["window"])
    return dict(begin=begin, end=end)


def _rms(x, w):
    """x / sqrt(mean x^2 + eps) * w, in 64 bits: what is stored is rounded next to borders."""
    x = x.double()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return y if w is None else y * w.double()


def _append(st):
    c, hd, sliding, dtype = st["case"], st["case"]["hd"], st["case"]["window"] > 0, _type(st["case"])
    axis = torch.tensor(_axis(c), device=st["q"].device)
    turns = axis.numel()
    freq = torch.pow(THETA[sliding], -2.0 * torch.arange(turns, device=axis.device).double() / hd).float().double()
    # angles in 64 bits: positions may be far
    angle = st["positions"].double()[axis].permute(1, 2, 0)[:, :, None, :] * freq
    cos = torch.nn.functional.pad(angle.cos(), (0, hd // 2 - turns), value=1.0)
    sin = torch.nn.functional.pad(angle.sin(), (0, hd // 2 - turns), value=0.0)

    def rope(y):
        a, b = y.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(dtype)

    cap = st["ck"].shape[2]
    rows = st["rows"].long()
    row = torch.where(rows >= 0, rows % cap if c["ring"] else rows, cap - 1)  # (the last row of a linear cache is spare)
    b = torch.arange(c["B"], device=rows.device)[:, None].expand_as(row)
    for_k, for_v = st["ck"].transpose(1, 2), st["cv"].transpose(1, 2)  # [B, rows, Hkv, hd]
    written = (rows >= 0)[:, :, None, None]
    for_k[b, row] = torch.where(written, rope(_rms(st["k"], st["kw"])), for_k[b, row])
    for_v[b, row] = torch.where(written, _rms(st["v"], None).to(dtype), for_v[b, row])
    return dict(q=rope(_rms(st["q"], st["qw"])), k=st["ck"], v=st["cv"])


def _positions(st, lens):
    """The position that each row of the cache holds, and whether it holds one."""
    rows = st["ck"].shape[2]
    row = torch.arange(rows, device=lens.device)[None, :]
    last = lens.long()[:, None] - 1
    at = last - (last - row) % rows if st["case"]["ring"] else row.expand(lens.numel(), -1)
    return at, (at >= 0) & (at <= last)


def _attend(st, q, keys_at, seen, distance):
    """q [B, Hkv, G, T, hd] against all rows; seen and distance [B, T, rows]."""
    c = st["case"]
    k = torch.where(keys_at[:, None, :, None], st["ck"].float(), 0.0)
    v = torch.where(keys_at[:, None, :, None], st["cv"].float(), 0.0)
    s = q.float() @ k.transpose(2, 3)[:, :, None]
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    if c["bias"]:
        s = s - st["slopes"].view(1, c["Hkv"], -1, 1, 1) * distance[:, None, None].float()
    seen = seen[:, None, None]
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top > -math.inf, top, 0.0))
    total = e.sum(-1, keepdim=True)
    return (e @ v[:, :, None]) / torch.where(total > 0, total, 1.0)


def _prefill(st):
    c, T = st["case"], st["case"]["T"]
    keys, held = _positions(st, st["start"] + T)
    held = held & (keys < st["lens"].long()[:, None])
    at = st["start"].long()[:, None] + torch.arange(T, device=keys.device)[None, :]
    if st["begin"] is None:
        end = at + 1
        begin = end - c["window"] if c["window"] else torch.zeros_like(at)
    else:
        begin, end = st["begin"], st["end"]
    seen = held[:, None] & (keys[:, None] >= begin[..., None]) & (keys[:, None] < end[..., None])
    q = st["q"].view(c["B"], T, c["Hkv"], -1, c["hd"]).permute(0, 2, 3, 1, 4)
    out = _attend(st, q, held, seen, (keys[:, None] - at[..., None]).abs())
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3).to(_type(c)).contiguous()


def _decode(st):
    c, lens = st["case"], st["lens"].long()
    keys, held = _positions(st, st["lens"])
    begin = lens - c["window"] if c["window"] else torch.zeros_like(lens)
    if st["begin"] is not None:
        begin = torch.maximum(begin, st["begin"].long())
    seen = held & (keys >= begin[:, None])
    q = st["q"].unflatten(1, (c["Hkv"], -1))[:, :, :, None]
    out = _attend(st, q, held, seen[:, None], (lens[:, None] - 1 - keys)[:, None])
    return out[:, :, :, 0].flatten(1, 2).to(_type(c))


def run(state):
    if own:
        return _run_own(state)
    return {"ranges": _ranges, "append": _append, "prefill": _prefill, "decode": _decode}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the work

def work(case):
    c = case
    B, T, mid, w = c["B"], c.get("T", 1), (c["lo"] + c["hi"]) / 2, c["window"]
    if c["op"] == "ranges":
        given = (c["doc"] > 0) + (c["span"] > 0)
        return dict(bytes=B * (8 * T + 4 * given * (mid + 0.75 * T)), flops=0)
    H, Hkv, hd, size = c["H"], c["Hkv"], c["hd"], 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "append":
        tokens = B * T
        kept = tokens * 0.75 if T > 1 else tokens
        return dict(bytes=size * hd * (2 * tokens * H + 4 * kept * Hkv) + 4 * tokens * (AXES + 1),
                    flops=tokens * (H + 2 * Hkv) * hd * 8)
    if c["op"] == "prefill":
        # the keys that a token sees on average: what precedes it in its document and window, half a span after it
        real = T if c["mask"] == "causal" else 0.875 * T
        docs, spans = c["mask"] in ("docs", "both"), c["mask"] in ("spans", "both")
        sees = lambda p: min(p + 1, w or p + 1, c["doc"] if docs else p + 1) + (c["span"] / 2 if spans else 0)  # noqa: E731
        pairs = sum(sees(mid + t) for t in range(int(real)))
        keys = min(mid + real, real + w) if w else mid + real
        return dict(bytes=B * size * hd * (2 * H * T + 2 * Hkv * keys), flops=4 * B * pairs * H * hd)
    keys = B * (min(mid, w) if w else mid) * (0.67 if c["begin"] else 1.0)
    return dict(bytes=size * hd * (2 * Hkv * keys + 2 * B * H), flops=4 * keys * H * hd)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "ranges":
        return None
    B, T, H, Hkv, hd, w = c["B"], c.get("T", 1), c["H"], c["Hkv"], c["hd"], c["window"]
    dev, rows = st["ck"].device, st["ck"].shape[2]
    if c["op"] == "append":
        half, axis = hd // 2, _axis(c)
        turns, out = len(axis), {}
        f = torch.tensor([THETA[w > 0] ** (-2.0 * j / hd) for j in range(turns)], device=dev).double()  # held in 32 bits
        turn = torch.stack([st["positions"][axis[j]].double() * f[j] for j in range(turns)], -1)[:, :, None]
        turn = torch.polar(torch.ones_like(turn), turn)
        for name, x, weight in (("q", st["q"], st["qw"]), ("k", st["k"], st["kw"]), ("v", st["v"], None)):
            x = x.double()
            y = x / (x.pow(2).sum(-1, keepdim=True) / hd + EPS).sqrt()
            if weight is not None:
                y = y * weight.double()
                z = torch.complex(y[..., :turns], y[..., half:half + turns]) * turn
                y = torch.cat([z.real, y[..., turns:half], z.imag, y[..., half + turns:]], -1)
            if name == "q":
                out[name] = y
                continue
            kept = torch.zeros(st["ck"].shape, dtype=torch.float64, device=dev)
            for b in range(B):
                at = st["rows"][b].long()
                fresh = (at >= 0).nonzero()[:, 0]
                kept[b][:, at[fresh] % rows] = y[b, fresh].transpose(0, 1)
            out[name] = kept
        return out
    slopes = st["slopes"].double() if c["bias"] else torch.zeros(H, dtype=torch.float64, device=dev)
    outs = []
    for b in range(B):
        n = int(st["lens"][b])
        first = int(st["start"][b]) if c["op"] == "prefill" else n - 1
        mine = torch.arange(first, first + T, device=dev)
        lowest = max(0, n - rows) if c["ring"] else 0
        if c["op"] == "decode":
            if w:
                lowest = max(lowest, n - w)
            if c["begin"]:
                lowest = max(lowest, int(st["begin"][b]))
        at = torch.arange(lowest, n, device=dev)
        hidden = at[None, :] > mine[:, None]
        if w:
            hidden = hidden | (at[None, :] <= mine[:, None] - w)
        if c["op"] == "prefill" and st["begin"] is not None:
            hidden = (at[None, :] < st["begin"][b, :, None]) | (at[None, :] >= st["end"][b, :, None])
        apart = (mine[:, None] - at[None, :]).abs().double()
        blind = hidden.all(1)
        per_head = []
        for h in range(H):
            g = h // (H // Hkv)
            q = (st["q"][b, :, h] if c["op"] == "prefill" else st["q"][b, h][None]).double()
            s = q @ st["ck"][b, g, at % rows].double().T
            if c["cap"]:
                s = torch.tanh(s / c["cap"]) * c["cap"]
            s = (s - apart * slopes[h]).masked_fill(hidden, -math.inf)
            s[blind] = 0.0
            o = torch.softmax(s, -1) @ st["cv"][b, g, at % rows].double()
            o[blind] = 0.0
            per_head.append(o)
        outs.append(torch.stack(per_head, 1))
    outs = torch.stack(outs)
    return outs if c["op"] == "prefill" else outs[:, 0]
