"""CPU oracle of the 8-bit cache and of attention with a sliding window and sinks.

TEST INFRASTRUCTURE, like oracle.paged_attention: float64 numpy, written from the
definitions, no code shared with the CUDA library.

Readings:
  * quantisation: e = max(-118, ceil(log2(amax / 448))), amax the largest finite magnitude
    of a row of head_dim values; a code is x * 2^-e rounded to the nearest e4m3 value, ties
    to the even code; a value that is not finite becomes the NaN code 0x7f;
  * a query at position p sees key j <= p iff there is no window (0), or j > p - window, or
    j < sinks.
"""

from __future__ import annotations

import math

import numpy as np

from .paged_attention import bf16_to_f64

E4M3_NAN = 0x7F


def e4m3_to_f64(codes) -> np.ndarray:
    """Decode e4m3 bytes (bias 7, no infinities, 0x7f and 0xff are NaN) to float64."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    sign = np.where(c >> 7, -1.0, 1.0)
    exp = (c >> 3) & 15
    frac = (c & 7).astype(np.float64)
    out = np.where(exp == 0, np.ldexp(frac, -9), np.ldexp(1.0 + frac / 8.0, exp - 7))
    return np.where((c & 127) == E4M3_NAN, np.nan, sign * out)


_POSITIVE = e4m3_to_f64(np.arange(127))     # ascending with the code


def f64_to_e4m3(x) -> np.ndarray:
    """Nearest e4m3 byte of finite x with |x| <= 448, ties to the even code."""
    x = np.asarray(x, np.float64)
    mag = np.abs(x)
    above = np.clip(np.searchsorted(_POSITIVE, mag), 0, 126)
    below = np.maximum(above - 1, 0)
    up, down = _POSITIVE[above] - mag, mag - _POSITIVE[below]
    code = np.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantise_rows(bits):
    """bf16 rows [..., D] (uint16 bits) -> (e4m3 bytes [..., D], scale bytes [...])."""
    x = bf16_to_f64(bits)
    finite = np.isfinite(x)
    amax = np.where(finite, np.abs(x), 0.0).max(-1)
    # smallest e >= -118 with amax <= 448 * 2^e
    frac, ex = np.frexp(amax)                              # amax = frac * 2^ex, 0.5 <= frac < 1
    e = np.where(amax > 0, ex - 9 + (frac > 0.875), -118)   # 448 = 0.875 * 2^9
    e = np.maximum(e, -118)
    code = f64_to_e4m3(np.ldexp(np.where(finite, x, 0.0), -e[..., None]))
    return np.where(finite, code, E4M3_NAN).astype(np.uint8), (e + 127).astype(np.uint8)


def dequantise_rows(codes, scale_bytes) -> np.ndarray:
    return np.ldexp(e4m3_to_f64(codes), np.asarray(scale_bytes, np.int64)[..., None] - 127)


def seen(num_keys: int, p: int, window: int, sinks: int) -> np.ndarray:
    """Which of num_keys keys a query at position p sees."""
    j = np.arange(num_keys)
    return (j <= p) & ((window == 0) | (j > p - window) | (j < sinks))


def attend(q, k, v, positions, window, sinks, scale):
    """One sequence: q [L, Hq, D], k and v [n, Hkv, D] float64, position of each query.

    Returns (out [L, Hq, D], lse [L, Hq], mass [L, Hq, D], spread [L, Hq]): mass is
    sum_j softmax_j |v_j| and spread the largest sum_d |q_d k_jd| * |scale| over visible keys,
    which error bounds are made of.  Values of keys that a query does not see are never
    touched.
    """
    L, hq, d = q.shape
    n, hkv, _ = k.shape
    g = hq // hkv
    out = np.zeros((L, hq, d))
    mass = np.zeros((L, hq, d))
    lse = np.full((L, hq), -np.inf)
    spread = np.zeros((L, hq))
    for r in range(L):
        m = seen(n, int(positions[r]), window, sinks)
        if not m.any():
            continue
        kk, vv = k[m], v[m]
        for h in range(hq):
            s = kk[:, h // g] @ q[r, h] * scale
            top = s.max()
            w = np.exp(s - top)
            tot = w.sum()
            w = w / tot
            out[r, h] = w @ vv[:, h // g]
            mass[r, h] = w @ np.abs(vv[:, h // g])
            lse[r, h] = top + math.log(tot)
            spread[r, h] = (np.abs(kk[:, h // g]) @ np.abs(q[r, h])).max() * abs(scale)
    return out, lse, mass, spread


def gather(pool, table, n, block_size):
    """Rows 0 .. n-1 of a sequence from a pool [num_blocks, block_size, ...]."""
    rows = [pool[int(table[j // block_size]), j % block_size] for j in range(n)]
    return np.stack(rows) if rows else np.zeros((0,) + pool.shape[2:], pool.dtype)
