"""Inputs, the fp64 definition and the tolerance of the scored-attention tests (numpy only).

Definition, per query row at position p of a sequence with L keys (q head h, kv head h / G):
  z_j = scale q.k_j;  z_j = cap tanh(z_j / cap);  z_j -= slope[h] |p - j|
  visible: j < L, j >= key_start, and (j < prefix or (j <= p and j > p - window))
  out = sum_j softmax(z)_j v_j over the visible j, 0 where there are none.

Tolerance. With A = sum_j softmax(z)_j |v_j| and u = 2^-24 (half an fp32 step, relative):
  * a score is off by at most dz = (D + 16) u scale max_j sum_d |q_d k_jd| (dot product in fp32, in
    any order) + 8 u max_j |z_j| (scale, bias, log2 domain: a few roundings of z, |bias| and |z|
    before the bias) + 2^-20 cap (the tanh, an absolute error of 2^-20);
  * a weight is then off by a factor e^(+-dz), the normaliser too, and each exponential by 2^-22:
    relative 2 (dz + 2^-21) (1 + dz), which moves the output by that times A;
  * sums over N keys in fp32, in any order, of numerator and normaliser: 2 (N + 16) u A;
  * bf16: the weights are rounded to bf16 before the product with V: 2^-8 A; the output is rounded
    once: 2^-8 (|out| + the above).  fp32: the output's last rounding is u |out|.
"""
from __future__ import annotations

import numpy as np

from paged_kv_cache_238_gb300 import workloads as W

U = 2.0 ** -24


def keys_seen(L, p, start, prefix, window):
    j = np.arange(L)
    near = (j <= p) & ((window == 0) | (j > p - window))
    return (j >= start) & ((j < prefix) | near)


class Case:
    """One batch over a pool. lens: keys per sequence; chunks: query rows per sequence (None:
    decode, one row at the last position). key_start: per row, prefix: per sequence."""

    def __init__(self, seed, lens, H_q, H_kv, D, BS=16, dtype="bf16", chunks=None, cap=0.0, slopes=None, window=0,
                 key_start=None, prefix=None, sharp=1.0, free_invisible=True):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, dtype=np.int32)
        S = len(self.lens)
        self.decode = chunks is None
        self.chunks = np.ones(S, dtype=np.int32) if chunks is None else np.asarray(chunks, dtype=np.int32)
        self.qsl = np.concatenate([[0], np.cumsum(self.chunks)]).astype(np.int32)
        T = int(self.qsl[-1])
        self.H_q, self.H_kv, self.D, self.BS, self.dtype = H_q, H_kv, D, BS, dtype
        self.cap, self.window = float(cap), int(window)
        self.slopes = None if slopes is None else np.asarray(slopes, dtype=np.float32)
        self.key_start = None if key_start is None else np.asarray(key_start, dtype=np.int32)
        self.prefix = None if prefix is None else np.asarray(prefix, dtype=np.int32)
        self.scale = 1.0 / float(np.sqrt(D))
        q = rng.standard_normal((T, H_q, D), dtype=np.float32) * np.float32(sharp)
        self.q = W.f32_to_bf16_bits(q) if dtype == "bf16" else q
        self.seen, self.keys, self.vals = [], [], []
        blocks = [-(-int(n) // BS) for n in self.lens]
        NB = 1 + sum(blocks) + 3
        ids = rng.permutation(np.arange(1, NB))
        self.k_cache = W._nan_like_pool((NB, H_kv, BS, D), dtype)
        self.v_cache = W._nan_like_pool((NB, H_kv, BS, D), dtype)
        self.table = np.zeros((S, max(1, max(blocks))), dtype=np.int32)
        at = 0
        for s in range(S):
            L, C = int(self.lens[s]), int(self.chunks[s])
            seen = np.zeros((C, L), dtype=bool)
            for r in range(C):
                p = L - C + r
                if p >= 0:
                    start = 0 if self.key_start is None else int(self.key_start[self.qsl[s] + r])
                    seen[r] = keys_seen(L, p, start, 0 if self.prefix is None else int(self.prefix[s]), self.window)
            any_row = seen.any(axis=0)
            k, v = W._draw(rng, (L, H_kv, D), dtype), W._draw(rng, (L, H_kv, D), dtype)
            mine = ids[at:at + blocks[s]].copy()
            at += blocks[s]
            for b in range(blocks[s]):  # pages that no row sees are given back: the null block
                if free_invisible and not any_row[b * BS:(b + 1) * BS].any():
                    mine[b] = 0
            self.table[s, :blocks[s]] = mine
            for j in np.flatnonzero(any_row):  # every other cell stays NaN
                self.k_cache[mine[j // BS], :, j % BS] = k[j]
                self.v_cache[mine[j // BS], :, j % BS] = v[j]
            self.seen.append(seen)
            self.keys.append(W.as_f64(k))
            self.vals.append(W.as_f64(v))

    def reference(self):
        """(out, tolerance), fp64 [T, H_q, D] each."""
        G = self.H_q // self.H_kv
        q = W.as_f64(self.q)
        out, tol = np.zeros(q.shape), np.zeros(q.shape)
        half = 2.0 ** -8 if self.dtype == "bf16" else U
        for s, seen in enumerate(self.seen):
            L, C = int(self.lens[s]), int(self.chunks[s])
            pos = L - C + np.arange(C)
            for h in range(self.H_q):
                K, V = self.keys[s][:, h // G], self.vals[s][:, h // G]
                qs = q[self.qsl[s]:self.qsl[s] + C, h]
                z = qs @ K.T * self.scale
                mag = np.abs(qs) @ np.abs(K).T * self.scale
                big = np.abs(z)
                if self.cap:
                    z = self.cap * np.tanh(z / self.cap)
                if self.slopes is not None:
                    bias = float(self.slopes[h]) * np.abs(pos[:, None] - np.arange(L)[None, :])
                    z = z - bias
                    big = np.maximum(big, bias)
                big = np.maximum(big, np.abs(z))
                for r in range(C):
                    vis = seen[r]
                    n = int(vis.sum())
                    if n == 0:
                        continue
                    w = np.exp(z[r, vis] - z[r, vis].max())
                    w /= w.sum()
                    o, A = w @ V[vis], w @ np.abs(V[vis])
                    dz = (self.D + 16) * U * mag[r, vis].max() + 8 * U * big[r, vis].max() + 2.0 ** -20 * self.cap
                    rel = 2 * (dz + 2.0 ** -21) * (1 + dz) + 2 * (n + 16) * U
                    if self.dtype == "bf16":
                        rel += 2.0 ** -8
                    out[self.qsl[s] + r, h] = o
                    tol[self.qsl[s] + r, h] = rel * A + half * (np.abs(o) + rel * A)
        return out, tol


def alibi(H_q):
    return [2.0 ** (-8.0 * (h + 1) / H_q) for h in range(H_q)]
