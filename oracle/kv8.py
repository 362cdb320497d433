"""fp64 oracle of the 8-bit paged KV cache (test infrastructure only).

Rows are kept as whole numbers of the method's own terms: an e4m3 value times
its block's power-of-two scale, one block per 16 slots of a KV head.  Nothing
here is shared with the CUDA library.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK, PAGE = 16, 64
TOP = 448.0


def round_e4m3(x) -> np.ndarray:
    """Nearest e4m3 value (ties to even, saturating at +-448, NaN kept)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), TOP)
    with np.errstate(divide="ignore"):
        e = np.where(a > 0, np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    step = 2.0 ** (np.clip(e, -6, 8) - 3)
    return np.copysign(np.round(a / step) * step, x)


def e4m3_of_byte(b) -> np.ndarray:
    """The e4m3 value of each byte, from the format: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    b = np.asarray(b, dtype=np.int64)
    sign, e, f = b >> 7, (b >> 3) & 15, b & 7
    v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((b & 0x7F) == 0x7F, np.nan, v)
    return np.where(sign == 1, -v, v)


def scale_of(rows) -> float:
    """The smallest power of two in [2^-40, 2^40] that brings every finite |x| within 448."""
    x = np.abs(np.asarray(rows, dtype=np.float64))
    x = x[np.isfinite(x)]
    top = x.max() if x.size else 0.0
    s = 2.0 ** -40
    while s < 2.0 ** 40 and TOP * s < top:
        s *= 2
    return s


def frequencies(rotary_dim, theta, factor=1.0, low=1.0, high=4.0, orig_len=0) -> np.ndarray:
    """Radians per position of each pair."""
    out = []
    for i in range(rotary_dim // 2):
        f = theta ** (-2.0 * i / rotary_dim)
        if factor != 1.0:
            if orig_len == 0:
                f /= factor
            else:
                turns = orig_len * f / (2 * math.pi)
                w = min(1.0, max(0.0, (turns - low) / (high - low)))
                f = w * f + (1 - w) * f / factor
        out.append(f)
    return np.array(out)


def rotate(x, pos, freq, interleaved) -> np.ndarray:
    """x [heads][hd] of one token."""
    y = np.array(x, dtype=np.float64)
    for i, f in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(freq))
        c, s = math.cos(pos * f), math.sin(pos * f)
        y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
    return y


class Rows:
    """One layer's keys or values of one sequence: e4m3 values [Hkv][slots][hd], scales [Hkv][blocks]."""

    def __init__(self, n_kv_heads, slots, hd):
        self.code = np.zeros((n_kv_heads, slots, hd))
        self.scale = np.full((n_kv_heads, (slots + BLOCK - 1) // BLOCK), 2.0 ** -40)

    def value(self, length) -> np.ndarray:
        s = np.repeat(self.scale, BLOCK, axis=1)[:, :length]
        return self.code[:, :length] * s[:, :, None]

    def append(self, length, new):
        """new [n][Hkv][hd] to slots length .. length + n - 1."""
        n = len(new)
        for blk in range(length // BLOCK, (length + n - 1) // BLOCK + 1):
            lo, hi = max(length, blk * BLOCK), min(length + n, (blk + 1) * BLOCK)
            for h in range(self.code.shape[0]):
                x = np.asarray(new)[lo - length:hi - length, h]
                s = scale_of(x)
                if blk * BLOCK < length:
                    s = max(s, self.scale[h, blk])
                    held = slice(blk * BLOCK, length)
                    self.code[h, held] = round_e4m3(self.code[h, held] * (self.scale[h, blk] / s))
                self.code[h, lo:hi] = round_e4m3(np.clip(x / s, -TOP, TOP))
                self.scale[h, blk] = s

    def commit(self, root, path):
        """Rows root + path[d - 1] -> root + d."""
        m = len(path)
        src = [root + s for s in path]
        came = [(self.code[:, t].copy(), self.scale[:, t // BLOCK].copy()) for t in src]
        for blk in sorted({(root + d) // BLOCK for d in range(1, m + 1)}):
            ds = [d for d in range(1, m + 1) if (root + d) // BLOCK == blk]
            for h in range(self.code.shape[0]):
                s = max(came[d - 1][1][h] for d in ds)
                if blk * BLOCK <= root:
                    s = max(s, self.scale[h, blk])
                    held = slice(blk * BLOCK, root + 1)
                    self.code[h, held] = round_e4m3(self.code[h, held] * (self.scale[h, blk] / s))
                for d in ds:
                    self.code[h, root + d] = round_e4m3(came[d - 1][0][h] * (came[d - 1][1][h] / s))
                self.scale[h, blk] = s


def attention(q, K, V, length, see, scale):
    """(o, a) of one sequence: q [n][H][hd], K, V [Hkv][length + n][hd], see [n][n] the new slots each
    token sees.  o [n][H][hd]; a the same sum with |v|, the size that rounding of the weights goes by."""
    n, H, hd = q.shape
    G = H // K.shape[0]
    o, a = np.zeros((n, H, hd)), np.zeros((n, H, hd))
    for j in range(n):
        at = np.concatenate([np.arange(length), length + np.flatnonzero(see[j])]).astype(int)
        if not len(at):
            continue
        for h in range(H):
            s = K[h // G][at] @ q[j, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            o[j, h] = p @ V[h // G][at]
            a[j, h] = p @ np.abs(V[h // G][at])
    return o, a
