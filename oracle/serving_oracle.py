"""Plain 64-bit definitions of the operators around the paged cache: rotary positions, the 8-bit
cache and attention with a sliding window.

TEST INFRASTRUCTURE ONLY, like the compression oracle beside it: numpy in fp64, one row, block or
token at a time, sharing no code with the library.
"""
from __future__ import annotations

import math

import numpy as np

# ------------------------------------------------------------------ rotary positions ---------


def rope_frequencies(rotary_dim, theta, scaling="none", factor=1.0, original_len=0, low=1.0, high=4.0):
    """(radians per position of each pair, factor on cos and sin)."""
    if scaling == "base":
        theta = theta * factor ** (rotary_dim / (rotary_dim - 2))
    out, size = [], 1.0
    for i in range(rotary_dim // 2):
        f = theta ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            size = 0.1 * math.log(factor) + 1.0
            ends = [rotary_dim * math.log(original_len / (n * 2 * math.pi)) / (2 * math.log(theta)) for n in (high, low)]
            lo, hi = max(math.floor(ends[0]), 0), min(math.ceil(ends[1]), rotary_dim - 1)
            ramp = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f * (1 - ramp) + f / factor * ramp
        elif scaling == "wavelength":
            turns = original_len * f / (2 * math.pi)
            mix = min(max((turns - low) / (high - low), 0.0), 1.0)
            f = (1 - mix) * f / factor + mix * f
        out.append(f)
    return np.array(out), size


def rope(x, positions, freqs, size, interleaved):
    """x [T, H, d] in fp64 -> rotated [T, H, d]."""
    half = len(freqs)
    y = x.copy()
    ang = positions.astype(np.float64)[:, None] * freqs
    c, s = (size * np.cos(ang))[:, None], (size * np.sin(ang))[:, None]
    ia, ib = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


# ------------------------------------------------------------------ 8-bit cache --------------


def e4m3_values():
    """The value of each of the 256 codes (NaN for 0x7F and 0xFF)."""
    v = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[code] = math.nan if code & 0x7F == 0x7F else (-x if code & 0x80 else x)
    return v


_VALUES = e4m3_values()


def e4m3_encode(x):
    """Nearest code of each value (ties to the even code); |x| <= 448 or NaN."""
    x = np.asarray(x, dtype=np.float64)
    pos = _VALUES[:0x7F]  # codes 0 .. 0x7E, increasing
    size = np.abs(x)
    hi = np.clip(np.searchsorted(pos, size), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = size - pos[lo], pos[hi] - size
    code = np.where(dlo < dhi, lo, np.where(dhi < dlo, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isnan(x), 0x7F, code + np.where(np.signbit(x), 0x80, 0))
    return code.astype(np.uint8)


def e4m3_decode(codes):
    return _VALUES[codes]


def block_scale(x):
    """Scale of a tile: the smallest power of two >= amax / 448 (finite values only), at least 2^-126."""
    fin = np.abs(x[np.isfinite(x)])
    amax = fin.max() if fin.size else 0.0
    if amax == 0:
        return 0.0
    e = -126
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def quantise(x, scale):
    x = np.where(np.isfinite(x), x, np.nan)
    return e4m3_encode(x / scale if scale > 0 else np.where(np.isnan(x), x, x * 0.0))


def append(codes, scales, layer, k, v, start, cached, tables, b):
    """codes uint8 [layers, NB, 2, H, b, d] and scales [layers, NB, 2, H], updated in place; k, v fp64
    [T, H, d]."""
    H = k.shape[1]
    for r in range(len(cached)):
        pos, end, t = int(cached[r]), int(cached[r] + start[r + 1] - start[r]), int(start[r])
        while pos < end:
            lo = pos % b
            n = min(b - lo, end - pos)
            blk = tables[r][pos // b]
            for i, x in enumerate((k, v)):
                for h in range(H):
                    new = x[t:t + n, h]
                    old = float(scales[layer, blk, i, h]) if lo else 0.0
                    s = max(old, block_scale(new))
                    tile = codes[layer, blk, i, h]
                    if lo and s > old:
                        tile[:lo] = e4m3_encode(e4m3_decode(tile[:lo]) * (old / s))
                    tile[lo:lo + n] = quantise(new, s)
                    scales[layer, blk, i, h] = s
            pos, t = pos + n, t + n


# ------------------------------------------------------------------ attention ----------------


def attention_row(q, k, v, scale, visible):
    """q [d], k and v [L, d] in fp64, visible bool [L] -> (output [d], sum of weight * |value| [d])."""
    t = np.nonzero(visible)[0]
    if len(t) == 0:
        return np.zeros_like(q), np.zeros_like(q)
    x = scale * (k[t] @ q)
    w = np.exp(x - x.max())
    w /= w.sum()
    return w @ v[t], w @ np.abs(v[t])


def window_visible(p, L, window, sinks):
    t = np.arange(L)
    return (t <= p) & ((t > p - window) | (t < sinks) | (window == 0))
