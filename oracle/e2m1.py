"""The 4-bit cache format in float64: E2M1 codes with E4M3 group scales.

Test infrastructure only (see the package docstring).

A (page, kv head) slice holds 16 tokens x 64 code bytes (dim 2i in the low
nibble of byte i), then 16 tokens x 8 E4M3 scale bytes, one for every 16 dims.
A value is the tensor's scale * group scale * E2M1(code). E2M1 (OCP 4-bit
floating point): sign, 2 exponent bits of bias 1, 1 mantissa bit, no infinities
or NaN. Encoding a group x of 16 values with tensor scale t:

    s    = E4M3(max |x| / t / 6)       to nearest even, at most 448
    code = E2M1(x / (t s))             to nearest even, at most 6
"""
from __future__ import annotations

import numpy as np

from . import e4m3

GROUP = 16
SLICE_BYTES = 1152
CODE_BYTES = 1024


def decode_closed_form(codes) -> np.ndarray:
    """Value of each nibble by the closed form: s = x >> 3, e = (x >> 1) & 3, m = x & 1;
    e == 0: m / 2, otherwise 2^(e-1) (1 + m/2)."""
    x = np.asarray(codes, dtype=np.int64)
    e, m = (x >> 1) & 3, (x & 1).astype(np.float64)
    mag = np.where(e == 0, m / 2.0, np.ldexp(1.0 + m / 2.0, e - 1))
    return np.where(x & 8, -mag, mag)


def lut() -> np.ndarray:
    return decode_closed_form(np.arange(16))


def nearest_even(a, grid) -> np.ndarray:
    """Index of the value of the ascending ``grid`` nearest to each a >= 0 (past
    its end: the last), ties to the even index."""
    a = np.asarray(a, np.float64)
    mid = (grid[1:] + grid[:-1]) / 2
    lo = np.searchsorted(mid, a, side="left")
    hi = np.searchsorted(mid, a, side="right")
    return np.where((lo != hi) & (lo % 2 == 1), hi, lo)


def encode(x, scale: float):
    """x [..., 128] float64 -> (codes uint8 [..., 64], scales uint8 [..., 8])."""
    g = np.asarray(x, np.float64).reshape(*np.shape(x)[:-1], 8, GROUP)
    fine = e4m3.lut()[:127]
    amax = np.abs(g).max(axis=-1)  # numpy's max keeps a NaN
    nan = np.isnan(amax)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        s8 = np.where(nan, 127, nearest_even(np.where(nan, 0, amax / scale / 6.0), fine))
        s = np.where(nan, 0.0, fine[np.where(nan, 0, s8)])
        q = np.where(s[..., None] > 0, np.abs(g) / (s[..., None] * scale), 0.0)
    c = nearest_even(q, lut()[:8]) + 8 * np.signbit(g)
    c = c.reshape(*np.shape(x)[:-1], 64, 2)
    return (c[..., 0] + 16 * c[..., 1]).astype(np.uint8), s8.astype(np.uint8)


def pack(codes, scales) -> np.ndarray:
    """codes [..., 16, 64], scales [..., 16, 8] -> slices uint8 [..., 1152]."""
    lead = codes.shape[:-2]
    return np.concatenate([codes.reshape(*lead, -1), scales.reshape(*lead, -1)], axis=-1)


def decode_slices(cache) -> np.ndarray:
    """uint8 [..., 1152] -> float64 [..., 16, 128], without the tensor's scale."""
    cache = np.asarray(cache, np.uint8)
    lead = cache.shape[:-1]
    codes = cache[..., :CODE_BYTES].reshape(*lead, 16, 64)
    s = e4m3.lut()[cache[..., CODE_BYTES:].reshape(*lead, 16, 8)]
    out = np.empty((*lead, 16, 128))
    out[..., 0::2] = lut()[codes & 15]
    out[..., 1::2] = lut()[codes >> 4]
    return (out.reshape(*lead, 16, 8, GROUP) * s[..., None]).reshape(*lead, 16, 128)


def paged_decode_attention(q, k_cache, v_cache, block_tables, context_lens, k_scale, v_scale,
                           sm_scale=None) -> np.ndarray:
    """q [B, Hq, 128] or [B, T, Hq, 128], caches [NB, Hkv, 1152]: float64 output of q's
    shape. New token i of T sees tokens 0 .. ctx - T + i (none: a zero row)."""
    q4 = np.asarray(q, np.float64).reshape(q.shape[0], -1, q.shape[-2], q.shape[-1])
    n_b, n_t, hq, d = q4.shape
    hkv = k_cache.shape[1]
    sm = sm_scale if sm_scale else 1.0 / np.sqrt(d)
    out = np.zeros_like(q4)
    for b in range(n_b):
        ctx = int(context_lens[b])
        pages = block_tables[b, :(ctx + 15) // 16].astype(np.int64)
        for h in range(hkv):
            k = k_scale * decode_slices(k_cache[pages, h]).reshape(-1, d)[:ctx]
            v = v_scale * decode_slices(v_cache[pages, h]).reshape(-1, d)[:ctx]
            for i in range(n_t):
                n = ctx - n_t + i + 1
                if n <= 0:
                    continue
                rows = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                s = sm * q4[b, i, rows] @ k[:n].T
                p = np.exp(s - s.max(axis=-1, keepdims=True))
                out[b, i, rows] = (p / p.sum(axis=-1, keepdims=True)) @ v[:n]
    return out.reshape(q.shape)
