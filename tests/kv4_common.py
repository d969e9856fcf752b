"""Pools, tables and references shared by the 4-bit cache's GPU tests."""

import numpy as np
import torch

from gemma_dual_geometry_gb300 import g4attn as G
from gemma_dual_geometry_gb300 import workloads as W
from oracle import g4_oracle as O
from oracle import kv4_oracle as K

from gpu_common import DEV, f64, geometry, params_of


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def bf16_normal(shape, seed):
    return W.normal(shape, seed, W.BF16)


class Pool:
    """A pool on the host and the device: random bytes (NaN scales among them) outside the rows that are
    written, a shuffled table of B sequences of at most ``most`` positions."""

    def __init__(self, geo, B, most, block_size, seed, k_exp=0, spare=2):
        self.geo, self.B, self.bs, self.k_exp = geo, B, block_size, k_exp
        self.hd, self.Hkv = geo["head_dim"], geo["n_kv_heads"]
        rng = np.random.default_rng(seed)
        self.per = max(1, -(-most // block_size))
        self.n = B * self.per + spare
        self.table = rng.permutation(self.n)[:B * self.per].reshape(B, self.per)
        self.data = rng.integers(0, 256, (self.n, self.Hkv, block_size // 16, 18 * self.hd), dtype=np.uint8)

    def slot(self, b, p):
        return int(self.table[b, p // self.bs]) * self.bs + p % self.bs

    def fill(self, lens, seed):
        """Unit rows at positions [0, lens[b]), by the oracle."""
        rng = np.random.default_rng(seed)
        kc, ks, vc, vs = K.record_offsets(self.hd)
        for b in range(self.B):
            n = int(lens[b])
            for kvh in range(self.Hkv):
                k = O.round_bf16(rng.standard_normal((n, self.hd)) * 2.0 ** self.k_exp)
                v = O.round_bf16(rng.standard_normal((n, self.hd)))
                kq, vq = K.quantise(k, self.k_exp), K.quantise(v)
                for p in range(n):
                    rec = self.data[self.table[b, p // self.bs], kvh, (p % self.bs) // 16]
                    m = p % 16
                    rec[kc[m, 0::2]] = kq[0][p, 0::2] | (kq[0][p, 1::2] << 4)
                    rec[ks[m, 0::16]] = kq[1][p]
                    rec[vc[m, 0::2]] = vq[0][p, 0::2] | (vq[0][p, 1::2] << 4)
                    rec[vs[m, 0::16]] = vq[1][p]
        return self

    def to_device(self):
        self.d = torch.from_numpy(self.data).to(DEV)
        self.d_table = i32(self.table)
        self.pools = G.kv4_pool_table(1)
        G.set_kv4_pool(self.pools, 0, self.d, self.geo["layer_type"], self.hd, self.Hkv, self.n, self.bs, self.k_exp)
        return self

    def rows(self, lens, cap):
        """K and V [B, Hkv, cap, hd] in float64, zero from lens[b] on."""
        k, v = (np.zeros((self.B, self.Hkv, cap, self.hd)) for _ in range(2))
        for b in range(self.B):
            n = min(int(lens[b]), cap)
            for kvh in range(self.Hkv):
                k[b, kvh, :n], v[b, kvh, :n] = K.read_rows(self.data, self.table[b], kvh, range(n), self.bs, self.k_exp)
        return k, v


def attention_and_scale(q, k, v, q_pos, lens, Hkv, geo):
    """The oracle's attention and the same weights on |v| (what relative errors of the weights act on);
    zeros for sequences without keys."""
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(q.shape[0]):
        if lens[b] < 1:
            continue
        one = slice(b, b + 1)
        for dst, vv in ((out, v), (mag, np.abs(v))):
            dst[one] = O.attention(q[one], k[one], vv[one], q_pos[one], lens[one], Hkv, geo["layer_type"],
                                   geo["window"], geo["attn_scale"])
    return out, mag


def assert_within(gpu, ref, mag, weights, what="", keys=0):
    """|gpu - ref| <= 2^-8 |ref| + weights * sum p |v| + keys * 2^-25: the output's rounding to bf16, the
    relative error ``weights`` of the probabilities, and where they are fp16 (decode, ``keys`` of them) what
    its subnormal range adds.  The largest probability of a row is formed as 2^4 or more, so the sum that
    divides is at least 2^4; a probability p and its product with its value's scale s are each rounded by
    at most 2^-25 there, which reaches the output as 2^-25 (s + 1) |code| / 2^4 per key; |code| <= 6 and
    s <= 1.6 (values of N(0, 1) rows stay below 6 * 1.6) make that at most 2^-25.  (1e-30: float32 has
    no weights below 2^-126.)"""
    gpu = np.asarray(gpu, np.float64)
    assert np.all(np.isfinite(gpu)), f"{what}: non-finite output"
    over = np.abs(gpu - ref) - (2.0 ** -8 * np.abs(ref) + weights * mag + keys * 2.0 ** -25 + 1e-30)
    assert (over <= 0).all(), f"{what}: {(over > 0).sum()} of {over.size} values off, worst by {over.max():.3e}"


__all__ = ["DEV", "G", "K", "O", "Pool", "W", "assert_within", "attention_and_scale", "bf16_normal", "f64", "geometry",
           "i32", "np", "params_of", "torch"]
