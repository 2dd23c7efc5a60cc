"""Plain fp64 reference for the 8-bit KV cache and the query / key norm with
rotation.

TEST INFRASTRUCTURE ONLY -- never imported by the product package.

A code stands for value(code) * scale.  e4m3 values come from the bits
(sign, 4 exponent bits with bias 7, 3 mantissa bits; 0x7f and 0xff are NaN);
int8 codes are two's complement.  Rounding is a search for the nearest entry
of the sorted table of values, ties to the even code.
"""
from __future__ import annotations

import math

import numpy as np

E4M3, INT8 = "e4m3", "int8"
QMAX = {E4M3: 448.0, INT8: 127.0}


def code_value(code: int, dtype: str) -> float:
    if dtype == INT8:
        return float(code - 256 if code > 127 else code)
    sign = -1.0 if code & 0x80 else 1.0
    e, m = (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    return sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))


TABLE = {d: np.array([code_value(c, d) for c in range(256)]) for d in (E4M3, INT8)}


def encode(y, dtype):
    """Codes (uint8) of float64 values already divided by their scale."""
    y = np.asarray(y, dtype=np.float64)
    pos = TABLE[dtype][:127 if dtype == E4M3 else 128]  # codes 0 .. 126 / 127: 0 .. qmax
    a = np.minimum(np.abs(np.where(np.isnan(y), 0.0, y)), pos[-1])
    hi = np.clip(np.searchsorted(pos, a), 1, len(pos) - 1)
    lo = hi - 1
    below, above = a - pos[lo], pos[hi] - a
    pick = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    neg = np.signbit(y)
    if dtype == INT8:
        c = np.where(neg, -pick, pick) & 0xff
        return np.where(np.isnan(y), 0, c).astype(np.uint8)
    c = pick | np.where(neg, 0x80, 0)
    nan = 0x7f | np.where(neg, 0x80, 0)
    return np.where(np.isnan(y), nan, c).astype(np.uint8)


def need(amax: float, dtype: str) -> float:
    """The smallest 2^e, e in [-100, 100], with amax <= qmax * 2^e."""
    e = -100
    while e < 100 and amax > QMAX[dtype] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def finite_max(rows) -> float:
    a = np.abs(np.asarray(rows, dtype=np.float64))
    a = a[np.isfinite(a)]
    return float(a.max()) if a.size else 0.0


class Cache:
    """Codes [NL, slots, H, D] and scales [NL, pages, H, P / block] of one pool."""

    def __init__(self, codes, scales, page_size, block, dtype):
        self.codes, self.scales = codes, scales
        self.P, self.block, self.dtype = page_size, block, dtype

    def at(self, slot):
        page, inside = divmod(slot, self.P)
        return page, inside // self.block, inside % self.block

    def append(self, layer, slots, rows):
        """Rows [n, H, D] of consecutive tokens into slots, block by block."""
        i = 0
        while i < len(slots):
            page, sub, inside = self.at(slots[i])
            n = 1
            while i + n < len(slots) and inside + n < self.block:
                n += 1
            first = slots[i] - inside
            for h in range(rows.shape[1]):
                new = rows[i:i + n, h]
                s = need(finite_max(new), self.dtype)
                if inside:
                    old = float(self.scales[layer, page, h, sub])
                    if old >= s:
                        s = old
                    else:
                        for r in range(first, slots[i]):
                            v = TABLE[self.dtype][self.codes[layer, r, h]]
                            self.codes[layer, r, h] = encode(v * old / s, self.dtype)
                self.codes[layer, slots[i]:slots[i] + n, h] = encode(new / s, self.dtype)
                self.scales[layer, page, h, sub] = s
            i += n

    def scale_of(self, layer, slots):
        """Scales [n, H] of slots, in float64."""
        slots = np.asarray(slots, dtype=np.int64)
        page, inside = slots // self.P, slots % self.P
        return self.scales[layer, page, :, inside // self.block].astype(np.float64)

    def rows(self, layer, slots):
        """Dequantised rows [n, H, D] in float64."""
        return TABLE[self.dtype][self.codes[layer, np.asarray(slots, dtype=np.int64)]] * \
            self.scale_of(layer, slots)[..., None]


def attention(q, k, v, scale, v_scale=None):
    """q [Hq, D], k and v [n, H, D] -> out [Hq, D], lse [Hq] and, for error bounds,
    sum_t p_t |v_t| [Hq, D], max_t sum_d |q_d k_td| * scale [Hq] and, given v's
    scales [n, H], max_t(p_t v_scale_t) sum_t |code_t| [Hq, D] (else zeros)."""
    Hq, D = q.shape
    n, H, _ = k.shape
    out, lse = np.zeros((Hq, D)), np.full(Hq, -np.inf)
    mass, size, floor = np.zeros((Hq, D)), np.zeros(Hq), np.zeros((Hq, D))
    for h in range(Hq if n else 0):
        g = h // (Hq // H)
        s = k[:, g] @ q[h] * scale
        m = s.max()
        p = np.exp(s - m)
        out[h] = p @ v[:, g] / p.sum()
        mass[h] = p @ np.abs(v[:, g]) / p.sum()
        lse[h] = m + math.log(p.sum())
        size[h] = (np.abs(k[:, g]) @ np.abs(q[h])).max() * abs(scale)
        if v_scale is not None:
            vs = v_scale[:, g]
            floor[h] = (p / p.sum() * vs).max() * np.abs(v[:, g] / vs[:, None]).sum(0)
    return out, lse, mass, size, floor


def norm_rope(x, weight, cos, sin, eps, interleaved):
    """x [heads, D]; weight [D] or None; cos, sin [rot / 2] -> [heads, D]."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    half = len(cos)
    out = y.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        out[:, a] = y[:, a] * cos[i] - y[:, b] * sin[i]
        out[:, b] = y[:, b] * cos[i] + y[:, a] * sin[i]
    return out
