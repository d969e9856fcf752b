"""The paged 4-bit cache through the stack driver: a four-layer stack (two
owning layers, two that read them) takes ragged prompts, decodes, loses and
admits sequences, against the float64 oracles; and its output next to the bf16
cache's differs by what 4 bits cost, no more."""

import numpy as np
import pytest

from gemma_dual_geometry_gb300 import build as g4build
from gemma_dual_geometry_gb300 import stack as S

from kv4_common import DEV, G, K, O, W, assert_within, attention_and_scale, bf16_normal, f64, i32, torch

pytestmark = pytest.mark.gpu

CFG = dict(B=5, H=4, Hkv=2, dtype=W.BF16, seed=0, types=[W.SLIDING, W.FULL, W.SLIDING, W.FULL], n_shared=2,
           geom={W.SLIDING: dict(head_dim=64, theta=1e4, rotary_fraction=1.0, window=24),
                 W.FULL: dict(head_dim=128, theta=1e6, rotary_fraction=0.25, window=0)})


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    g4build.build()
    G.lib()
    yield
    assert G.g4_take_device_error() == 0


def test_paged_stack_lifecycle():
    B, H, Hkv = CFG["B"], CFG["H"], CFG["Hkv"]
    st = S.PagedAttnStack(CFG, max_len=160, n_blocks=26, block_size=32, device=DEV)
    assert st.src == [-1, -1, 0, 1] and set(st.pools) == {0, 1}
    w = [[W.norm_weight(g["head_dim"], 10 * l + i) for i in range(2)] for l, g in enumerate(st.geo)]
    held = [[[] for _ in range(B)] for _ in range(2)]  # rows of the owning layers, as stored
    lens = np.zeros(B, int)
    plan = [(40, [40, 3, 0, 17, 29]), (1, [41, 4, 0, 18, 30]), (1, [42, 5, 1, 0, 31]), (30, [60, 35, 31, 9, 31]),
            (1, [61, 36, 32, 10, 32]), (1, [62, 0, 33, 11, 33])]
    for step, (T, want) in enumerate(plan):
        positions, slots = st.assign(i32(want), T)
        pos = positions.cpu().numpy()
        assert np.array_equal(st.lens.cpu().numpy(), want)   # the pool suffices
        for l, g in enumerate(st.geo):
            hd = g["head_dim"]
            q = bf16_normal((B, T, H, hd), 1000 * step + l)
            k, v = ((bf16_normal((B, T, Hkv, hd), 1000 * step + 50 * i + l) for i in (1, 2)) if st.owns(l) else (None, None))
            dev = [None if x is None else x.to(DEV) for x in (q, k, v)]
            q_out, out = torch.empty_like(dev[0]), torch.empty_like(dev[0])
            st.append(l, *dev, w[l][0].to(DEV), w[l][1].to(DEV) if st.owns(l) else None, T, q_out)
            if T > 1:
                st.prefill_attn(l, q_out, T, out)
            else:
                st.decode_attn(l, q_out, out)
            # the same with the oracles
            th, fr, eps = g["theta"], g["rotary_fraction"], g["eps"]
            qn = O.round_bf16(O.normrope_q(f64(q), f64(w[l][0]), pos, hd, th, fr, eps))
            rows = held[l if st.owns(l) else st.src[l]]
            if st.owns(l):
                kn, vn = (O.round_bf16(x) for x in O.normrope_kv(f64(k), f64(v), f64(w[l][1]), pos, hd, th, fr, eps))
                kn, vn = K.values(*K.quantise(kn)), K.values(*K.quantise(vn))
                for b in range(B):
                    del rows[b][want[b]:]
                    rows[b] += [(kn[b, t], vn[b, t]) for t in range(max(0, want[b] - lens[b]))]
                    assert len(rows[b]) == want[b]
            for b in range(B):
                fresh = want[b] - lens[b]
                if fresh <= 0:
                    continue
                kk, vv = (np.stack([r[i] for r in rows[b]], 1)[None] for i in (0, 1))
                at = (lens[b] + np.arange(fresh))[None]
                ref, mag = attention_and_scale(qn[b:b + 1, :fresh], kk, vv, at, np.array([want[b]]), Hkv, g)
                assert_within(f64(out[b:b + 1, :fresh]), ref, mag, 2.0 ** -8 if T == 1 else 2.0 ** -7,
                              f"step {step} layer {l} sequence {b}", keys=want[b] if T == 1 else 0)
        lens = np.array(want)
    # what is read back is what was written
    for l in (0, 1):
        hd = st.geo[l]["head_dim"]
        k, v = (torch.empty((B, Hkv, 70, hd), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        st.gather(l, i32(np.zeros(B)), 70, k, v)
        for b in range(B):
            for i, got in ((0, k), (1, v)):
                ref = np.zeros((Hkv, 70, hd))
                for p, r in enumerate(held[l][b]):
                    ref[:, p] = r[i]
                assert np.array_equal(f64(got[b]), ref)


@pytest.mark.parametrize("raw", [False, True])
def test_assign_on_a_stream_of_its_own(raw):
    """All that assign() does comes after what its stream still has to do: here two assignments that wait on it."""
    st = S.PagedAttnStack(CFG, max_len=160, n_blocks=26, block_size=32, device=DEV)
    want = [i32(x) for x in ([9, 40, 0, 33, 2], [12, 45, 6, 33, 0])]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    on = side.cuda_stream if raw else side
    st.assign(want[0], 40, stream=on)
    positions, slots = st.assign(want[1], 7, stream=on)
    torch.cuda.synchronize()
    assert torch.equal(st.start, want[0]) and torch.equal(st.lens, want[1])
    t = torch.arange(7, device=DEV)
    at = want[0][:, None] + t
    assert torch.equal(positions, torch.where(at < want[1][:, None], at, -1).int())
    assert torch.equal(slots >= 0, positions >= 0)


def test_stored_rows_are_the_bf16_caches_quantised():
    """The same tokens through g4_kv_append_normrope and g4_kv4_append_normrope: equal q, and the pool stands
    for the bf16 cache's rows quantised, bit for bit."""
    B, T, H, Hkv, hd, cap = 2, 96, 8, 2, 256, 128
    p = G.layer_params(W.FULL, hd, H, Hkv, 0, 1e6, 0.25)
    q, k, v = (bf16_normal((B, T, n, hd), s).to(DEV) for n, s in ((H, 1), (Hkv, 2), (Hkv, 3)))
    qw, kw = W.norm_weight(hd, 4).to(DEV), W.norm_weight(hd, 5).to(DEV)
    pos = i32(np.arange(T)[None, :].repeat(B, 0))
    ck, cv = (torch.zeros((B, Hkv, cap, hd), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = G.cache_table(1)
    G.set_cache(table, 0, ck, cv, W.FULL, hd, Hkv, cap, B, W.BF16)
    q1 = torch.empty_like(q)
    G.g4_kv_append_normrope(p, table, 0, q, k, v, qw, kw, pos, B, T, q1)
    data = torch.zeros(G.kv4_pool_bytes(4, Hkv, 64, hd), dtype=torch.uint8, device=DEV)
    pools = G.kv4_pool_table(1)
    G.set_kv4_pool(pools, 0, data, W.FULL, hd, Hkv, 4, 64)
    blocks = i32([[2, 0], [1, 3]])
    slots = blocks.gather(1, (pos // 64).long()) * 64 + pos % 64
    q2 = torch.empty_like(q)
    G.g4_kv4_append_normrope(p, pools, 0, q, k, v, qw, kw, pos, slots.int(), B, T, q2)
    assert torch.equal(q1, q2)
    k4, v4 = (torch.empty((B, Hkv, T, hd), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    G.g4_kv4_gather(p, pools, 0, blocks, 2, i32([0, 0]), i32([T, T]), B, T, k4, v4)
    for got, full in ((k4, ck[:, :, :T]), (v4, cv[:, :, :T])):
        want = K.values(*K.quantise(f64(full)))
        assert np.array_equal(f64(got), want)
