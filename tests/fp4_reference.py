"""Definitions and tolerances of the rotation and 4-bit pool tests (numpy only, fp64).

The pool: y = x / factor; per 16 dims scale = e4m3(max |y| / 6), code = e2m1(y / scale), both to nearest with ties to
even; value = code scale factor. A page of 16 tokens is 16 rows of codes (even dim in the low half of a byte), then 16
rows of scales. Bytes are compared exactly: with inputs that are numbers of the call's type every border is decided by
exact arithmetic (fp64 holds the border products, and the rotated k is rounded to the type first; its fp64 value is
within 2^-50 of exact, so it rounds the same way unless it lies that near to a border of the type).

Rotation, per element a c + b s in fp32 (one product rounded, one fused): off by at most 2 u (|a c| + |b s|), u = 2^-24,
then one rounding to the type, half a step: 2^-8 (bf16) or 2^-24 (fp32) of the magnitude.

Attention, with A = sum_j softmax(z)_j |v_j|, n visible keys:
  * a score: the dot product in fp32 in any order, each addition rounded or cut: dz = 2 (D + 16) u scale sum_d |q_d k_d|,
    and 8 u |z| for its scaling;  tensor cores: the query row in fp16 after a power of two that brings its largest
    magnitude to [1, 2): at most 2^-25 of that (2 ^ ceil) lost per element: scale qmax 2^-24 sum_d |k_d| more;
  * weights are off by e^(+-dz) and 2^-21 for the exponential, numerator and normaliser alike: 2 (dz + 2^-21) (1 + dz) A;
  * sums over n keys in fp32, cut or rounded: 4 (n + 16) u A;
  * bf16 queries: weights rounded to fp16 (2^-11), those below 2^-14 of the largest to 2^-25: 2^-11 A + n 2^-25 max |v|;
    where they are rounded to bf16 instead (CUDA cores do not round): covered by 2^-11 as well, since none is;
  * fp32 queries on the tensor cores: q and the weights as sums of two halves. A row's largest magnitude lies in
    [2^14, 2^15), so q_d is off by max(2^-22 |q_d|, 2^-25), the latter 2^-39 qmax: 4 u sum |q_d k_d| of the 2 (D + 16) u
    above, and scale qmax 2^-39 sum_d |k_d| more. The largest weight is 2^7 at least, so a weight w of a sum l is off by
    max(2^-22 w, 2^-25), 2^-25 being 2^-32 l at most: with the 2^-22 of the exponential, 2^-21, and n 2^-32 max |v|;
  * the output rounded once: 2^-8 (bf16) or u.
"""
from __future__ import annotations

import numpy as np

from paged_kv_cache_238_gb300 import workloads as W

U = 2.0 ** -24
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_bytes(x):
    """fp64 >= 0 -> bytes, nearest, ties to even, at most 448."""
    x = np.minimum(np.asarray(x, dtype=np.float64), 448.0)
    e = np.floor(np.log2(np.maximum(x, 2.0 ** -6)))
    n = np.rint(x / 2.0 ** (e - 3))  # 8..16 from 2^-6 on, 0..8 below
    return np.where(n >= 8, (e + 7) * 8 + (n - 8), n).astype(np.int64).astype(np.uint8)


def e4m3_values(b):
    b = b.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    return np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m * 2.0 ** -9)


def quantise(x, factor=1.0):
    """x fp64 [..., D] -> (codes uint8 [..., D], scale bytes [..., D / 16])."""
    y = (x / factor).reshape(*x.shape[:-1], -1, 16)
    sb = e4m3_bytes(np.abs(y).max(-1) / 6.0)
    s = e4m3_values(sb)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        a = np.where(s > 0, np.abs(y) / np.where(s > 0, s, 1), 0.0)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    mag = np.minimum(np.rint(a / step) * step, 6.0)
    codes = np.searchsorted(GRID, mag) + 8 * ((y < 0) | ((y == 0) & np.signbit(y)))
    return np.where(s > 0, codes, 0).astype(np.uint8).reshape(x.shape), sb


def to_pool(x, factor=1.0):
    """x fp64 [NB, H, BS, D] -> pool bytes [NB, H, BS, 9 D / 16]."""
    NB, H, BS, D = x.shape
    codes, scales = quantise(x, factor)
    packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
    pages = np.concatenate([packed.reshape(NB, H, BS // 16, 8 * D), scales.reshape(NB, H, BS // 16, D)], axis=-1)
    return np.ascontiguousarray(pages).reshape(NB, H, BS, 9 * D // 16)


def from_pool(pool, factor=1.0):
    """pool bytes [NB, H, BS, 9 D / 16] -> values fp64 [NB, H, BS, D]."""
    NB, H, BS, row = pool.shape
    D = row * 16 // 9
    pages = pool.reshape(NB, H, BS // 16, 9 * D)
    packed = pages[..., :8 * D].reshape(NB, H, BS, D // 2)
    scales = e4m3_values(pages[..., 8 * D:]).reshape(NB, H, BS, D // 16)
    codes = np.stack([packed & 15, packed >> 4], axis=-1).reshape(NB, H, BS, D)
    val = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return val * np.repeat(scales, 16, axis=-1) * factor  # (scale byte 0x7F reads as 480 here; no key has it)


def rotate(x, cs, interleaved):
    """x [T, H, D], cs [T, R] -> (rotated, sum of the magnitudes of each element's products), fp64."""
    R = cs.shape[1]
    c, s = cs[:, None, :R // 2], cs[:, None, R // 2:]
    out, mag = x.copy(), np.zeros_like(x)
    ia, ib = (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (np.arange(R // 2), np.arange(R // 2, R))
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia], mag[..., ib] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return out, mag


def rotate_tolerance(out, mag, dtype):
    half = 2.0 ** -8 if dtype == "bf16" else U
    return 2 * U * mag + half * (np.abs(out) + 2 * U * mag)


def rounded(x, dtype):
    """fp64 -> the type's numbers (through fp32, nearest), as fp64."""
    x = x.astype(np.float32)
    return W.as_f64(W.f32_to_bf16_bits(x)) if dtype == "bf16" else x.astype(np.float64)


class Case:
    """One batch over 4-bit pools. lens: keys per sequence; chunks: query rows per sequence (None: decode). Cells that hold
    no key have codes of 6 and scales of NaN (0x7F); block 0 too."""

    def __init__(self, seed, lens, H_q, H_kv, D, BS=16, dtype="bf16", chunks=None, k_scale=1.0, v_scale=1.0, sharp=1.0,
                 extra_blocks=3):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, dtype=np.int32)
        S = len(self.lens)
        self.decode = chunks is None
        self.chunks = np.ones(S, dtype=np.int32) if chunks is None else np.asarray(chunks, dtype=np.int32)
        self.qsl = np.concatenate([[0], np.cumsum(self.chunks)]).astype(np.int32)
        self.H_q, self.H_kv, self.D, self.BS, self.dtype = H_q, H_kv, D, BS, dtype
        self.k_scale, self.v_scale, self.scale = float(k_scale), float(v_scale), 1.0 / float(np.sqrt(D))
        q = rng.standard_normal((int(self.qsl[-1]), H_q, D), dtype=np.float32) * np.float32(sharp)
        self.q = W.f32_to_bf16_bits(q) if dtype == "bf16" else q
        blocks = [-(-int(n) // BS) for n in self.lens]
        NB = 1 + sum(blocks) + extra_blocks
        ids = rng.permutation(np.arange(1, NB))
        self.table = np.zeros((S, max(1, max(blocks, default=1))), dtype=np.int32)
        self.pools, self.values = [], []
        held = np.zeros((NB, BS), dtype=bool)
        at = 0
        for s in range(S):
            mine = ids[at:at + blocks[s]]
            at += blocks[s]
            self.table[s, :blocks[s]] = mine
            for b, blk in enumerate(mine):
                held[blk, :min(BS, int(self.lens[s]) - b * BS)] = True
        for f in (self.k_scale, self.v_scale):
            x = rng.standard_normal((NB, H_kv, BS, D)) * f
            pool = to_pool(x, f)
            pages = pool.reshape(NB, H_kv, BS // 16, 9 * D)
            dead = ~held.reshape(NB, BS // 16, 16)[:, None].repeat(H_kv, axis=1)
            pages[..., :8 * D][np.repeat(dead, D // 2, axis=-1)] = 0x77
            pages[..., 8 * D:][np.repeat(dead, D // 16, axis=-1)] = 0x7F
            self.pools.append(pool)
            self.values.append(from_pool(pool, f))

    def keys(self, s):
        L, BS = int(self.lens[s]), self.BS
        ids = self.table[s, :-(-L // BS)]
        return [v[ids].transpose(1, 0, 2, 3).reshape(self.H_kv, -1, self.D)[:, :L] for v in self.values]

    def reference(self):
        """(out, tolerance), fp64 [T, H_q, D] each."""
        q = W.as_f64(self.q)
        out, tol = np.zeros(q.shape), np.zeros(q.shape)
        half = 2.0 ** -8 if self.dtype == "bf16" else U
        for s in range(len(self.lens)):
            L, C, r0 = int(self.lens[s]), int(self.chunks[s]), int(self.qsl[s])
            if L == 0 or C == 0:
                continue
            K, V = self.keys(s)
            vis = np.arange(L)[None, :] <= (L - C + np.arange(C))[:, None]
            for h in range(self.H_q):
                k, v = K[h // (self.H_q // self.H_kv)], V[h // (self.H_q // self.H_kv)]
                qs = q[r0:r0 + C, h]
                z = np.where(vis, qs @ k.T * self.scale, -np.inf)
                mag = np.where(vis, np.abs(qs) @ np.abs(k).T * abs(self.scale), 0).max(1)
                dz = 2 * (self.D + 16) * U * mag + 8 * U * np.abs(np.where(vis, z, 0)).max(1)
                if self.dtype == "bf16":
                    dz = dz + abs(self.scale) * np.abs(qs).max(1) * 2.0 ** -24 * np.abs(k).sum(1).max()
                else:
                    dz = dz + abs(self.scale) * np.abs(qs).max(1) * 2.0 ** -39 * np.abs(k).sum(1).max()
                w = np.exp(z - z.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                o, A, n = w @ v, w @ np.abs(v), vis.sum(1)
                rel = 2 * (dz + 2.0 ** -21) * (1 + dz) + 4 * (n + 16) * U + (2.0 ** -11 if self.dtype == "bf16" else 0.0)
                err = rel[:, None] * A + n[:, None] * (2.0 ** -25 if self.dtype == "bf16" else 2.0 ** -32) * np.abs(v).max()
                out[r0:r0 + C, h] = o
                tol[r0:r0 + C, h] = err + half * (np.abs(o) + err)
        return out, tol
