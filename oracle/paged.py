"""Paged key/value cache in fp64, one sequence, head and row at a time: the definition that the
appending and attending kernels are tested against.  e4m3 numbers come from their bit patterns."""
import math

import numpy as np

from .attention import forward_decode


def e4m3_values():
    """The 256 e4m3 numbers by code: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f is NaN."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        if c & 127 == 127:
            x = math.nan
        out[c] = -x if c & 128 else x
    return out


E4M3 = e4m3_values()
_POS = E4M3[:127]   # 0 .. 448, increasing; neighbouring codes alternate in their last bit


def e4m3_encode(x):
    """Codes (uint8) of fp64 values: nearest, ties to the even code, beyond 448 saturated, NaN to NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.minimum(np.searchsorted(_POS, a), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def e4m3_scale(amax):
    """The smallest power of two s with amax <= 448 s, at least 2^-117."""
    s = 2.0 ** -117
    while s * 448.0 < amax:
        s *= 2.0
    return s


def rotate(x, pos, cos, sin, interleaved):
    """x [T, d] at positions pos [T]; pairs (i, i + r/2), or (2i, 2i + 1)."""
    half = cos.shape[1]
    y = np.array(x, dtype=np.float64)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cos[pos, i].astype(np.float64), sin[pos, i].astype(np.float64)
        y[:, a] = x[:, a] * c - x[:, b] * s
        y[:, b] = x[:, b] * c + x[:, a] * s
    return y


def sequence_keys(pool, page_table, b, L):
    """[Hkv, L, d] of sequence b, in order, from pool values [n_pages, Hkv, page, d]."""
    page = pool.shape[2]
    rows = [pool[page_table[b, j // page], :, j % page] for j in range(L)]
    return np.stack(rows, 1) if rows else np.zeros((pool.shape[1], 0, pool.shape[3]))


def forward_paged(q, k_pool, v_pool, page_table, key_lens, new_lens, scale, causal):
    """O [B,Hq,Nq,d] and lse [B,Hq,Nq]; query i of sequence b stands at key_lens[b] - new_lens[b] + i."""
    B, Hq, Nq, d = q.shape
    Hkv = k_pool.shape[1]
    O, lse = np.zeros(q.shape), np.full((B, Hq, Nq), -np.inf)
    for b in range(B):
        L, n = int(key_lens[b]), int(new_lens[b])
        if L == 0 or n == 0:
            continue
        k, v = (np.repeat(sequence_keys(x, page_table, b, L), Hq // Hkv, 0)[None] for x in (k_pool, v_pool))
        O[b, :, :n], lse[b, :, :n] = (x[0] for x in forward_decode(q[b: b + 1, :, :n], k, v, scale, causal))
    return O, lse
