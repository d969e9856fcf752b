"""Cases that measure the operators of the paged KV cache in 4 bits.

The cache holds keys and values as e2m1 codes with one e4m3 scale per 16
consecutive elements of a row, in blocks of ``block`` positions that a table
gives to requests.  Five operators work on it:

  blocks   gives a batch's requests blocks of a pool as their lengths change,
           and says where each new token goes (``slots``);
  append   norm + RoPE of q and k, norm of v, k and v written in 4 bits at
           their slots;
  gather   reads positions of requests back as bf16;
  decode   attention of one query per request over its blocks;
  prefill  causal attention of a chunk of new tokens over its request's blocks.

``run`` computes them in plain torch operations where ``own`` is false and
calls the library where it is true.  A group of 16 positions of one kv head is
a record of 18 * hd bytes: K codes, K scales, V codes, V scales, each in the
order ``pack`` writes them.
"""

import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
EPS = 1e-6
# theta and the rotated part of a head on sliding and on full layers
THETA = {True: 1e4, False: 1e6}
ROTATED = {True: 1.0, False: 0.25}


# ------------------------------------------------------------------ the cases

def listed():
    full = dict(H=8, Hkv=2, hd=512, window=0)
    slide = dict(H=8, Hkv=2, hd=256, window=512)
    return [
        # one decode step of a batch of 64: every request grows by a token, a few
        # end and a few are admitted with a single token
        dict(name="blocks step 64", op="blocks", B=64, T=1, block=64, lo=1024, hi=8192),
        # a step that also takes in prompts of up to 2048 tokens
        dict(name="blocks chunk 96x2048", op="blocks", B=96, T=2048, block=16, lo=1, hi=6000),
        # the new token of 64 requests on a sliding layer
        dict(name="append step 64 sliding", op="append", B=64, T=1, block=64, lo=1024, hi=8192, kexp=0, **slide),
        # a prompt chunk of 8 requests on a full layer
        dict(name="append 8x2048 full", op="append", B=8, T=2048, block=64, lo=0, hi=2048, kexp=0, **full),
        # a short request read back, as for moving it to another pool
        dict(name="gather 1x700", op="gather", B=1, rows=700, block=16, lo=700, hi=700, kexp=-2, H=4, Hkv=2, hd=128, window=0),
        # the contexts of 8 requests read back
        dict(name="gather 8x4096 full", op="gather", B=8, rows=4096, block=64, lo=2048, hi=4096, kexp=0, **full),
        # the smallest decode: one short request, where latency counts
        dict(name="decode 1x333", op="decode", B=1, block=16, lo=333, hi=333, kexp=0, H=8, Hkv=1, hd=128, window=0),
        # a serving batch on a sliding layer: 512 keys of each request
        dict(name="decode 64 sliding", op="decode", B=64, block=64, lo=1024, hi=8192, kexp=0, **slide),
        # the same batch on a full layer
        dict(name="decode 64 full", op="decode", B=64, block=64, lo=1024, hi=8192, kexp=0, **full),
        # few requests of a long context
        dict(name="decode 4x131072 full", op="decode", B=4, block=128, lo=131072, hi=131072, kexp=0, **full),
        # a chunk of 256 tokens after contexts of up to 4000 on a sliding layer
        dict(name="prefill 4x256 sliding", op="prefill", B=4, T=256, block=32, lo=500, hi=4000, kexp=1, **slide),
        # a chunk of 2048 tokens after a context as long on a full layer
        dict(name="prefill 2x2048 full", op="prefill", B=2, T=2048, block=64, lo=1500, hi=2048, kexp=0, **full),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is spread evenly over lo .. hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["blocks", "append", "gather", "decode", "decode", "prefill"])
    block = rng.choice([16, 32, 64, 128])
    if op == "blocks":
        T = rng.choice([1, 1, _log(rng, 2, 2048)])
        hi = _log(rng, 64, 20000)
        return dict(op=op, B=_log(rng, 1, 96 if T > 256 else 1000), T=T, block=block, lo=rng.randrange(0, hi), hi=hi)
    hd = rng.choice([64, 128, 256, 512])
    group = rng.choice([g for g in (1, 2, 4, 8) if g * hd <= 2048])
    Hkv = rng.choice([1, 2, 2, 4])
    c = dict(op=op, block=block, kexp=rng.choice([0, 0, -3, 2]), H=group * Hkv, Hkv=Hkv, hd=hd,
             window=rng.choice([0, _log(rng, 1, 1500)]))
    # a drawn case stays below the largest listed one
    if op == "append":
        T = rng.choice([1, _log(rng, 2, 2048)])
        most = max(1, (1 << 26) // (T * (c["H"] + 2 * Hkv) * hd))
        c.update(B=_log(rng, 1, min(256, most)), T=T, lo=0, hi=_log(rng, 1, 20000))
    elif op == "gather":
        rows = _log(rng, 1, 8000)
        most = max(1, (1 << 24) // (rows * Hkv * hd))
        c.update(B=_log(rng, 1, min(64, most)), rows=rows, lo=rows // 2, hi=rows)
    elif op == "decode":
        hi = _log(rng, 1, 30000)
        most = max(1, (1 << 28) // (hi * Hkv * hd))
        c.update(B=_log(rng, 1, min(200, most)), lo=rng.randrange(0, hi + 1), hi=hi)
    else:
        T, hi = _log(rng, 1, 1500), _log(rng, 1, 4000)
        most = max(1, (1 << 26) // (c["H"] * T * (T + hi)))
        c.update(B=_log(rng, 1, min(8, most)), T=T, lo=rng.randrange(0, hi + 1), hi=hi)
    return c


# ------------------------------------------------------------------ the format

def quantise(x, exp):
    """Codes (0..15) and scale bytes of bf16-valued rows x [..., hd], each divided by 2**exp first."""
    y = torch.ldexp(x.double(), torch.tensor(-exp, device=x.device)).unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0).float().to(torch.float8_e4m3fn)
    s = scale.double()
    m = torch.where(s > 0, y.abs() / torch.where(s > 0, s, 1.0), 0.0)
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = code + 8 * (y < 0).to(torch.uint8)
    return code.flatten(-2), scale.squeeze(-1).view(torch.uint8)


def values(code, scale, exp):
    """float32 values of codes [..., hd] and scale bytes [..., hd / 16]."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    v = grid[(code & 7).int()] * (1.0 - 2.0 * (code >> 3).float())
    s = scale.contiguous().view(torch.float8_e4m3fn).float() * 2.0 ** exp
    return (v.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def pack(kc, ks, vc, vs):
    """The records [..., block / 16, 18 * hd] of codes [..., block, hd] and scales [..., block, hd / 16]."""
    lead, hd = kc.shape[:-2], kc.shape[-1]
    n, p, x = kc.shape[-2] // 16, hd // 64, len(lead) + 1

    def order(t, shape, to):
        t = t.reshape(*lead, n, *shape)
        return t.permute(*range(x), *(x + i for i in to)).reshape(*lead, n, -1)

    # a K row m = (r, g) of a group, its element ((piece, w), t, byte, nibble)
    k = kc.reshape(*lead, n, 2, 8, p, 4, 4, 2, 2)
    k = order(k[..., 0] | k[..., 1] << 4, (2, 8, p, 4, 4, 2), (2, 1, 4, 0, 3, 5))
    s = order(ks, (2, 8, p, 4), (2, 1, 3, 0))
    # a V row m = (ih, t, il), its element ((piece, w), g, nibble)
    v = vc.reshape(*lead, n, 2, 4, 2, p, 4, 8, 2)
    v = order(v[..., 0] | v[..., 1] << 4, (2, 4, 2, p, 4, 8), (3, 5, 1, 0, 2, 4))
    z = order(vs, (2, 4, 2, p, 4), (3, 1, 4, 0, 2))
    return torch.cat([k, s, v, z], -1)


def unpack(rec):
    """Codes and scales (kc, ks, vc, vs) of records [..., block / 16, 18 * hd]."""
    lead, n, hd = rec.shape[:-2], rec.shape[-2], rec.shape[-1] // 18
    p, x = hd // 64, len(lead) + 1

    def order(t, shape, to):
        t = t.reshape(*lead, n, *shape)
        return t.permute(*range(x), *(x + i for i in to)).contiguous()

    k, s, v, z = rec.split([8 * hd, hd, 8 * hd, hd], -1)
    k = order(k, (p, 8, 4, 2, 4, 2), (3, 1, 0, 4, 2, 5))
    v = order(v, (p, 8, 4, 2, 2, 4), (3, 2, 4, 0, 5, 1))
    kc = torch.stack([k & 15, k >> 4], -1).reshape(*lead, 16 * n, hd)
    vc = torch.stack([v & 15, v >> 4], -1).reshape(*lead, 16 * n, hd)
    ks = order(s, (p, 8, 4, 2), (3, 1, 0, 2)).reshape(*lead, 16 * n, hd // 16)
    vs = order(z, (p, 4, 4, 2, 2), (3, 1, 4, 0, 2)).reshape(*lead, 16 * n, hd // 16)
    return kc, ks, vc, vs


# ------------------------------------------------------------------ the inputs

def _unit(shape, gen):
    """bf16 rows of unit mean square, as a cache is appended."""
    x = torch.randn(shape, generator=gen, device=DEVICE)
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)).bfloat16()


def _lengths(c, gen, n):
    return torch.randint(c["lo"], c["hi"] + 1, (n,), generator=gen, device=DEVICE, dtype=torch.int32)


def _tables(c, gen, most):
    """A table that deals a shuffled pool out to the requests, `most` positions each; entries past them are -1."""
    B, block = c["B"], c["block"]
    per = max(1, -(-int(most.max()) // block))
    need = (most.long() + block - 1) // block
    used = torch.arange(per, device=DEVICE)[None, :] < need[:, None]
    n = B * per + 3
    table = torch.randperm(n, generator=gen, device=DEVICE)[: B * per].view(B, per)
    return torch.where(used, table, -1).int(), n


def _slots(table, positions, block):
    b = table.long().gather(1, (positions.clamp(min=0).long() // block))
    return torch.where((positions >= 0) & (b >= 0), b * block + positions % block, -1).int()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    st = dict(case=c)
    if c["op"] == "blocks":
        B, T, block = c["B"], c["T"], c["block"]
        old = _lengths(c, gen, B)
        kind = torch.rand(B, generator=gen, device=DEVICE)
        grow = torch.randint(1, T + 1, (B,), generator=gen, device=DEVICE, dtype=torch.int32)
        old = torch.where(kind < 0.1, 0, old)                       # admitted now
        new = torch.where((kind > 0.9) & (old > 0), 0, old + grow)  # ended
        per = -(-(c["hi"] + T) // block)
        n = B * per + 7
        used = torch.arange(per, device=DEVICE)[None, :] < ((old + block - 1) // block)[:, None]
        ids = torch.randperm(n, generator=gen, device=DEVICE).int()
        table = torch.where(used, ids[: B * per].view(B, per), -1)
        taken = torch.zeros(n, dtype=torch.bool, device=DEVICE)
        taken[table[used].long()] = True
        left = ids[~taken[ids.long()]]
        free = torch.full((n,), -1, dtype=torch.int32, device=DEVICE)
        free[: left.numel()] = left
        # one pool in three has too few blocks left for all requests
        count = left.numel() if seed % 3 else left.numel() // 8
        st.update(old=old, new=new.int(), table=table.contiguous(), free=free, per=per, n=n,
                  count=torch.tensor([count], dtype=torch.int32, device=DEVICE))
    elif c["op"] == "append":
        B, T, H, Hkv, hd = c["B"], c["T"], c["H"], c["Hkv"], c["hd"]
        start = _lengths(c, gen, B)
        fresh = torch.randint(max(1, T // 2), T + 1, (B,), generator=gen, device=DEVICE, dtype=torch.int32)
        lens = start + fresh
        table, n = _tables(c, gen, lens)
        t = torch.arange(T, device=DEVICE, dtype=torch.int32)[None, :]
        positions = torch.where(t < fresh[:, None], start[:, None] + t, -1).int()
        weight = lambda: 1.0 + 0.1 * torch.randn(hd, generator=gen, device=DEVICE)  # noqa: E731
        row = lambda heads: torch.randn((B, T, heads, hd), generator=gen, device=DEVICE).bfloat16()  # noqa: E731
        st.update(q=row(H), k=row(Hkv), v=row(Hkv), qw=weight(), kw=weight(), positions=positions,
                  slots=_slots(table, positions, c["block"]), start=start, lens=lens, table=table, n=n,
                  data=torch.zeros((n, Hkv, c["block"] // 16, 18 * hd), dtype=torch.uint8, device=DEVICE))
    else:
        B, H, Hkv, hd, block = c["B"], c["H"], c["Hkv"], c["hd"], c["block"]
        lens = _lengths(c, gen, B)
        if c["op"] == "prefill":
            st["start"] = lens
            lens = lens + c["T"]
        table, n = _tables(c, gen, lens)
        # rows that no request uses hold any bytes
        data = torch.randint(0, 256, (n, Hkv, block // 16, 18 * hd), generator=gen, device=DEVICE, dtype=torch.uint8)
        share = max(1, (1 << 26) // (Hkv * block * hd))
        k_gain = 2.0 ** c["kexp"]
        for i in range(0, n, share):
            shape = (min(share, n - i), Hkv, block, hd)
            kc, ks = quantise(_unit(shape, gen).float() * k_gain, c["kexp"])
            vc, vs = quantise(_unit(shape, gen).float(), 0)
            data[i:i + share] = pack(kc, ks, vc, vs)
        st.update(lens=lens, table=table, n=n, data=data)
        if c["op"] == "decode":
            st["q"] = (_unit((B, H, hd), gen) / k_gain).bfloat16()
        elif c["op"] == "prefill":
            st["q"] = (_unit((B, c["T"], H, hd), gen) / k_gain).bfloat16()
        else:
            st["start"] = torch.randint(0, 1 + c["rows"] // 4, (B,), generator=gen, device=DEVICE, dtype=torch.int32)
    if own:
        st["kept"] = _kept(st)  # handles, workspaces and output buffers that a program keeps; no data is laid out
    return st


# ------------------------------------------------------------------ the library's calls

def _kept(st):
    from gemma_dual_geometry_gb300 import g4attn as G
    c, z = st["case"], {}
    empty = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device=DEVICE)  # noqa: E731
    if c["op"] == "blocks":
        B, T, i32 = c["B"], c["T"], torch.int32
        z.update(lens=empty(B, dtype=i32), count=empty(1, dtype=i32), positions=empty(B, T, dtype=i32),
                 slots=empty(B, T, dtype=i32))
        return z
    kind = G.G4_SLIDING if c["window"] else G.G4_FULL
    z["params"] = p = G.layer_params(kind, c["hd"], c["H"], c["Hkv"], c["window"], THETA[c["window"] > 0],
                                     ROTATED[c["window"] > 0], EPS, 1.0, -1, G.G4_BF16)
    z["pools"] = G.kv4_pool_table(1)
    G.set_kv4_pool(z["pools"], 0, st["data"], kind, c["hd"], c["Hkv"], st["n"], c["block"], c["kexp"])
    z["per"] = st["table"].shape[1]
    if c["op"] in ("append", "gather"):
        rows = c["T"] if c["op"] == "append" else c["rows"]
        z.update(k=empty(c["B"], c["Hkv"], rows, c["hd"]), v=empty(c["B"], c["Hkv"], rows, c["hd"]))
    if c["op"] == "append":
        z["q"] = torch.empty_like(st["q"])
    if c["op"] in ("decode", "prefill"):
        z["most"] = most = z["per"] * c["block"]
        z["bytes"] = (G.g4_kv4_decode_workspace_size(p, c["B"], most) if c["op"] == "decode"
                      else G.g4_kv4_prefill_workspace_size(p, c["B"], c["T"], most))
        z["ws"] = torch.zeros(max(16, z["bytes"]), dtype=torch.uint8, device=DEVICE)
        z["out"] = torch.empty_like(st["q"])
    return z


def _run_own(st):
    from gemma_dual_geometry_gb300 import g4attn as G
    c, z = st["case"], st["kept"]
    if c["op"] == "blocks":
        G.g4_kv4_assign_blocks(c["B"], c["T"], c["block"], st["n"], st["per"], st["old"], st["new"], st["free"],
                               st["count"], st["table"], z["lens"], z["count"], z["positions"], z["slots"])
        return dict(table=st["table"], free=st["free"], lens=z["lens"], count=z["count"], positions=z["positions"],
                    slots=z["slots"])
    if c["op"] == "append":
        G.g4_kv4_append_normrope(z["params"], z["pools"], 0, st["q"], st["k"], st["v"], st["qw"], st["kw"],
                                 st["positions"], st["slots"], c["B"], c["T"], z["q"])
        G.g4_kv4_gather(z["params"], z["pools"], 0, st["table"], z["per"], st["start"], st["lens"], c["B"], c["T"],
                        z["k"], z["v"])
        return dict(q=z["q"], k=z["k"], v=z["v"])
    if c["op"] == "gather":
        G.g4_kv4_gather(z["params"], z["pools"], 0, st["table"], z["per"], st["start"], st["lens"], c["B"], c["rows"],
                        z["k"], z["v"])
        return dict(k=z["k"], v=z["v"])
    if c["op"] == "decode":
        G.g4_kv4_attn_decode(z["params"], z["pools"], 0, st["q"], st["table"], z["per"], st["lens"], c["B"], z["most"],
                             z["out"], z["ws"], z["bytes"])
        return z["out"]
    G.g4_kv4_attn_prefill(z["params"], z["pools"], 0, st["q"], st["table"], z["per"], st["start"], st["lens"], c["B"],
                          c["T"], z["most"], z["out"], z["ws"], z["bytes"])
    return z["out"]


# ------------------------------------------------------------------ the plain forms

def _blocks(st):
    c, dev = st["case"], st["old"].device
    T, block, per = c["T"], c["block"], st["per"]
    table, free = st["table"].clone(), st["free"].clone()
    old = st["old"].long().clamp(0, per * block)
    new = torch.minimum(st["new"].long().clamp(0, per * block), old + T)
    have, want = (old + block - 1) // block, (new + block - 1) // block
    entry = torch.arange(per, device=dev)[None, :]
    # blocks given back go to the end of the free list, in the order of requests
    count = st["count"].long()
    back = (entry >= want[:, None]) & (entry < have[:, None])
    place = torch.where(back, count + back.flatten().cumsum(0).view_as(back) - 1, free.numel())
    free = torch.cat([free, free[:1]]).scatter(0, place.flatten(), table.flatten())[:-1]
    # and are taken from its end, requests first come, first served
    there = count + back.sum()
    need = (want - have).clamp(min=0)
    upto = need.cumsum(0)
    granted = (need == 0) | (upto <= there)
    take = (entry >= have[:, None]) & (entry < want[:, None]) & granted[:, None]
    nth = (upto - need)[:, None] + entry - have[:, None]
    table = torch.where(take, free[(there - 1 - nth).clamp(0, free.numel() - 1)], table)
    lens = torch.where(granted, new, old)
    at = old[:, None] + torch.arange(T, device=dev)[None, :]
    fresh = at < lens[:, None]
    positions = torch.where(fresh, at, -1)
    block_of = table.long().gather(1, (at // block).clamp(max=per - 1))
    slots = torch.where(fresh, block_of * block + at % block, -1)
    left = there - (need * granted).sum()
    return dict(table=table, free=free, lens=lens.int(), count=left.int(), positions=positions.int(), slots=slots.int())


def _rms(x, w):
    """x / sqrt(mean x^2 + eps) * w, in 64 bits: what is stored is rounded next to borders."""
    x = x.double()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return y if w is None else y * w.double()


def _rope(y, positions, sliding):
    """rotate_half of rows y [B, T, heads, hd] by their positions, in 64 bits (angles of far positions)."""
    hd = y.shape[-1]
    j = torch.arange(hd // 2, device=y.device)
    freq = torch.pow(THETA[sliding], -2.0 * j.double() / hd).float().double()
    freq = torch.where(j < int(hd * ROTATED[sliding] / 2), freq, 0.0)
    angle = (positions.double()[..., None] * freq)[:, :, None, :]
    a, b = y.chunk(2, -1)
    return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)


def _append(st):
    c, sliding = st["case"], st["case"]["window"] > 0
    q = _rope(_rms(st["q"], st["qw"]), st["positions"], sliding).bfloat16()
    k = _rope(_rms(st["k"], st["kw"]), st["positions"], sliding).bfloat16()
    v = _rms(st["v"], None).bfloat16()
    written = (st["slots"] >= 0)[:, :, None, None]
    k = torch.where(written, values(*quantise(k, c["kexp"]), c["kexp"]), 0.0)
    v = torch.where(written, values(*quantise(v, 0), 0), 0.0)
    return dict(q=q, k=k.transpose(1, 2).bfloat16().contiguous(), v=v.transpose(1, 2).bfloat16().contiguous())


def _read(st, first, count):
    """float32 K and V [B, Hkv, n, hd] of `count` blocks of each request from block first[b] on, and their positions."""
    c, block = st["case"], st["case"]["block"]
    at = first[:, None].long() + torch.arange(count, device=first.device)[None, :]
    ids = torch.where(at < st["table"].shape[1], st["table"].long().gather(1, at.clamp(max=st["table"].shape[1] - 1)), -1)
    rec = st["data"][ids.clamp(min=0)]  # [B, count, Hkv, block / 16, 18 hd]
    kc, ks, vc, vs = (t.transpose(1, 2).flatten(2, 3) for t in unpack(rec))
    positions = (at[:, :, None] * block + torch.arange(block, device=first.device)).flatten(1)
    there = (positions < st["lens"][:, None])[:, None, :, None]
    k = torch.where(there, values(kc, ks, c["kexp"]), 0.0)
    v = torch.where(there, values(vc, vs, 0), 0.0)
    return k, v, positions


def _gather(st):
    c, block = st["case"], st["case"]["block"]
    first = st["start"] // block
    k, v, positions = _read(st, first, -(-c["rows"] // block) + 1)
    at = (st["start"] % block).long()[:, None] + torch.arange(c["rows"], device=first.device)[None, :]
    at = at[:, None, :, None].expand(-1, c["Hkv"], -1, c["hd"])
    return dict(k=k.gather(2, at).bfloat16(), v=v.gather(2, at).bfloat16())


def _softmax_v(scores, seen, v):
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = torch.where(seen, torch.exp(scores - torch.where(top > -math.inf, top, 0.0)), 0.0)
    total = e.sum(-1, keepdim=True)
    return (e @ v) / torch.where(total > 0, total, 1.0)


def _decode(st):
    c, block, lens = st["case"], st["case"]["block"], st["lens"]
    low = (lens - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(lens)
    count = min(st["table"].shape[1], -(-c["window"] // block) + 1) if c["window"] else st["table"].shape[1]
    k, v, positions = _read(st, low // block, count)
    q = st["q"].float().unflatten(1, (c["Hkv"], -1))
    seen = ((positions >= low[:, None]) & (positions < lens[:, None]))[:, None, None, :]
    return _softmax_v(q @ k.transpose(2, 3), seen, v).flatten(1, 2).bfloat16()


def _prefill(st):
    c, block, start, T = st["case"], st["case"]["block"], st["start"], st["case"]["T"]
    low = (start - c["window"] + 1).clamp(min=0) if c["window"] else torch.zeros_like(start)
    count = st["table"].shape[1]
    if c["window"]:
        count = min(count, -(-(c["window"] + T) // block) + 1)
    k, v, positions = _read(st, low // block, count)
    q = st["q"].float().view(c["B"], T, c["Hkv"], -1, c["hd"]).permute(0, 2, 3, 1, 4)
    at = start[:, None] + torch.arange(T, device=start.device)[None, :]
    gap = at[:, :, None] - positions[:, None, :]
    seen = gap >= 0
    if c["window"]:
        seen = seen & (gap < c["window"])
    out = _softmax_v(q @ k.transpose(2, 3)[:, :, None], seen[:, None, None], v[:, :, None])
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3).bfloat16().contiguous()


def run(state):
    if own:
        return _run_own(state)
    return {"blocks": _blocks, "append": _append, "gather": _gather, "decode": _decode, "prefill": _prefill}[
        state["case"]["op"]](state)


# ------------------------------------------------------------------ the work

def work(case):
    c = case
    B, mid = c["B"], (c["lo"] + c["hi"]) / 2
    if c["op"] == "blocks":
        T, block = c["T"], c["block"]
        ids = B * (T + 1) / 2 / block
        return dict(bytes=B * 8 + ids * 8 + B * 4 + B * T * 8, flops=0)
    H, Hkv, hd, w = c["H"], c["Hkv"], c["hd"], c["window"]
    row = 9 * hd / 16  # bytes of one K or V row
    if c["op"] == "append":
        tokens = B * c["T"]
        kept = tokens * 0.75 if c["T"] > 1 else tokens
        nbytes = tokens * (4 * H * hd + 8) + kept * (4 * Hkv * hd + 2 * Hkv * row) + tokens * 4 * Hkv * hd
        return dict(bytes=nbytes, flops=tokens * (H + 2 * Hkv) * hd * 8)
    if c["op"] == "gather":
        return dict(bytes=B * Hkv * c["rows"] * 4 * hd + B * Hkv * 2 * row * min(c["rows"], mid), flops=0)
    if c["op"] == "decode":
        keys = B * (min(mid, w) if w else mid)
        return dict(bytes=keys * Hkv * 2 * row + B * H * hd * 4, flops=keys * H * hd * 4)
    T = c["T"]
    pairs = sum(min(mid + t + 1, w) if w else mid + t + 1 for t in range(T))
    keys = min(mid + T, T + w - 1) if w else mid + T
    return dict(bytes=B * keys * Hkv * 2 * row + B * T * H * hd * 4, flops=B * pairs * H * hd * 4)


# ------------------------------------------------------------------ the definition in 64 bits

def _element(data, block_ids, position, block, head, hd, is_v):
    """The stored number of each element of the rows at `position` of blocks `block_ids` (same shape), without the
    exponent of k: the byte's place is computed from the position and the element."""
    d = torch.arange(hd, device=data.device)
    m, group = position % 16, position % block // 16
    m, group = m[..., None], group[..., None]
    piece, w = d // 64, d // 16 % 4
    if is_v:
        t, i = m % 8 // 2, m % 2 + m // 8 * 2
        code_at = 9 * hd + piece * 512 + (d % 16 // 2 * 4 + t) * 16 + i * 4 + w
        scale_at = 17 * hd + piece * 64 + t * 16 + w * 4 + i
    else:
        g, r = m % 8, m // 8
        code_at = piece * 512 + (g * 4 + d % 16 // 4) * 16 + r * 8 + w * 2 + d % 4 // 2
        scale_at = 8 * hd + piece * 64 + g * 8 + w * 2 + r
    byte = data[block_ids[..., None], head, group, code_at]
    nibble = (byte >> (4 * (d % 2)).to(torch.uint8)) & 15
    sign, e, man = nibble >> 3, (nibble >> 1 & 3).double(), (nibble & 1).double()
    code = torch.where(e == 0, man / 2, torch.exp2(e - 1) * (1 + man / 2)) * torch.where(sign > 0, -1.0, 1.0)
    s = data[block_ids[..., None], head, group, scale_at]
    se, sm = (s >> 3 & 15).double(), (s & 7).double()
    return code * torch.where(se == 0, sm * 2.0 ** -9, torch.exp2(se - 7) * (1 + sm / 8))


def _to_grid(x):
    """x [..., hd] in 64 bits as the cache stands for it, by distances to the numbers that codes and scales can hold."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    byte = torch.arange(127, device=x.device)
    e, man = (byte // 8).double(), (byte % 8).double()
    held = torch.where(e == 0, man * 2.0 ** -9, torch.exp2(e - 7) * (1 + man / 8))

    def nearest(v, table):
        up = torch.searchsorted(table, v.contiguous()).clamp(1, table.numel() - 1)
        below, above = v - table[up - 1], table[up] - v
        return torch.where((above < below) | ((above == below) & (up % 2 == 0)), up, up - 1)

    y = x.unflatten(-1, (-1, 16))
    # the largest number over 6, compared exactly: both sides times 6
    scale = held[nearest(y.abs().amax(-1), held * 6)][..., None]
    # |x| / scale against the grid, compared exactly: the grid times the scale
    mids, evens = (grid[1:] + grid[:-1]) / 2, torch.arange(7, device=x.device) % 2 == 0
    size, border = y.abs()[..., None], (scale[..., None] * mids)
    code = (torch.where(evens, size > border, size >= border) & (border > 0)).sum(-1)
    return (grid[code] * scale * torch.where(y < 0, -1.0, 1.0)).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "blocks":
        return None
    dev, hd, H, Hkv, w, block = st["data"].device, c["hd"], c["H"], c["Hkv"], c["window"], c["block"]
    if c["op"] == "append":
        half = hd // 2
        turns = int(hd * ROTATED[w > 0] / 2)
        out = {}
        for name, x, weight in (("q", st["q"], st["qw"]), ("k", st["k"], st["kw"]), ("v", st["v"], None)):
            x = x.double()
            y = x / (x.pow(2).sum(-1, keepdim=True) / hd + EPS).sqrt()
            if weight is not None:
                y = y * weight.double()
                f = torch.tensor([THETA[w > 0] ** (-2.0 * j / hd) for j in range(turns)], device=dev).double()
                z = torch.complex(y[..., :turns], y[..., half:half + turns])
                phase = st["positions"].double()[:, :, None, None] * f
                z = z * torch.polar(torch.ones_like(phase), phase)
                y = torch.cat([z.real, y[..., turns:half], z.imag, y[..., half + turns:]], -1)
            if name == "q":
                out["q"] = y
            else:
                e = 2.0 ** (c["kexp"] if name == "k" else 0)
                y = _to_grid(y.bfloat16().double() / e) * e
                y = y * (st["slots"] >= 0)[:, :, None, None]
                out[name] = y.transpose(1, 2)
        return out
    lens, k_gain = st["lens"].long(), 2.0 ** c["kexp"]
    outs = []
    for b in range(c["B"]):
        n = int(lens[b])
        start = int(st["start"][b]) if "start" in st else max(0, n - w) if w else 0
        if c["op"] == "gather":
            first, end = start, start + c["rows"]
        elif c["op"] == "decode":
            first, end = start, n
        else:
            first, end = max(0, start - w + 1) if w else 0, start + c["T"]
        at = torch.arange(first, end, device=dev)
        in_use = at < n
        ids = st["table"][b].long()[(at // block).clamp(max=st["table"].shape[1] - 1)].clamp(min=0)
        per_head = []
        for h in range(Hkv):
            k = torch.where(in_use[:, None], _element(st["data"], ids, at, block, h, hd, False) * k_gain, 0.0)
            v = torch.where(in_use[:, None], _element(st["data"], ids, at, block, h, hd, True), 0.0)
            if c["op"] == "gather":
                per_head.append((k, v))
                continue
            g = H // Hkv
            if c["op"] == "decode":
                q = st["q"][b, h * g:(h + 1) * g].double()
                per_head.append(torch.softmax(q @ k.T, -1) @ v if n else torch.zeros_like(q))
                continue
            rows = torch.arange(start, start + c["T"], device=dev)
            hidden = at[None, :] > rows[:, None]
            if w:
                hidden = hidden | (at[None, :] <= rows[:, None] - w)
            for x in range(h * g, (h + 1) * g):
                s = (st["q"][b, :, x].double() @ k.T).masked_fill(hidden, -math.inf)
                per_head.append(torch.softmax(s, -1) @ v)
        if c["op"] == "gather":
            outs.append((torch.stack([k for k, _ in per_head]), torch.stack([v for _, v in per_head])))
        elif c["op"] == "decode":
            outs.append(torch.cat(per_head))
        else:
            outs.append(torch.stack(per_head, 1))
    if c["op"] == "gather":
        return dict(k=torch.stack([k for k, _ in outs]), v=torch.stack([v for _, v in outs]))
    return torch.stack(outs)
