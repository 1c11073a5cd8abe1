"""Rotated key/value cache in float64 (test oracle only).

A head vector x of length d is held as the absmax codes of u = H_d diag(s) x /
sqrt(d), one scale for the whole vector: a = max|u|, scale = a / qmax, q =
clamp(rint(u / scale), -qmax, qmax), qmax = 2^(bits-1) - 1, stored as q +
2^(bits-1) (4 bits: two per byte, low nibble first).  A vector that is not
finite has a NaN scale and codes 0.  H is the Sylvester matrix, so the rotation
is orthogonal: scores of rotated queries with rotated keys are the scores of
the originals, and an average of rotated values is the rotated average.

Positions: sequence s owns tokens cu[s] .. cu[s + 1] of a call, the last of
its lens[s] positions; position p lives in page table[s][p // page_size].

Everything is written as loops over tokens and heads with numpy matrix
products; there is no tiling, no online softmax and no packed arithmetic.
"""
from __future__ import annotations

import numpy as np

from .hadamard import sylvester


def places(cu, lens, tokens: int):
    """(sequence, position) of every token, (None, None) for a token of no sequence."""
    out = [(None, None)] * tokens
    for s in range(len(lens)):
        n = int(cu[s + 1]) - int(cu[s])
        for i in range(n):
            t = int(cu[s]) + i
            if 0 <= t < tokens:
                out[t] = (s, int(lens[s]) - n + i)
    return out


def slot(table, pages: int, page_size: int, s: int, p: int):
    """(page, offset) of position p of sequence s, or None where it does not exist."""
    if p < 0 or p // page_size >= table.shape[1]:
        return None
    page = int(table[s, p // page_size])
    return (page, p % page_size) if 0 <= page < pages else None


def rope(x, angles, interleaved: bool):
    """x [..., d] turned by angles [pairs]; pairs (j, j + pairs) or (2j, 2j + 1)."""
    y = np.array(x, dtype=np.float64)
    for j, a in enumerate(np.asarray(angles, dtype=np.float64)):
        p, q = (2 * j, 2 * j + 1) if interleaved else (j, j + len(angles))
        y[..., p] = x[..., p] * np.cos(a) - x[..., q] * np.sin(a)
        y[..., q] = x[..., p] * np.sin(a) + x[..., q] * np.cos(a)
    return y


def angles(inv_freq, pos: int, t: int, positions=None, axis=None):
    """Angle of every pair of token t at sequence position pos."""
    f = np.asarray(inv_freq, dtype=np.float64)
    if positions is None:
        return pos * f
    p = np.atleast_2d(np.asarray(positions, dtype=np.float64))
    ax = np.zeros(len(f), dtype=int) if axis is None else np.asarray(axis, dtype=int)
    return np.array([p[a, t] * v if 0 <= a < p.shape[0] else 0.0 for a, v in zip(ax, f)])


def rotate(x, signs):
    """H diag(signs) x / sqrt(d) along the last axis."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    s = np.ones(d) if signs is None else np.asarray(signs, dtype=np.float64)
    return (x * s) @ sylvester(d).astype(np.float64) / np.sqrt(d)


def unrotate(u, signs):
    """diag(signs) H u / sqrt(d) along the last axis."""
    u = np.asarray(u, dtype=np.float64)
    d = u.shape[-1]
    s = np.ones(d) if signs is None else np.asarray(signs, dtype=np.float64)
    return u @ sylvester(d).astype(np.float64) / np.sqrt(d) * s


def quantize(u, bits: int):
    """(q, scale, t) of vectors along the last axis; t = u / scale before rounding."""
    qmax = 2 ** (bits - 1) - 1
    a = np.abs(u).max(axis=-1)
    s = a / qmax
    fine = np.isfinite(s) & (s > 0)
    with np.errstate(invalid="ignore"):
        t = np.where(fine[..., None], u / np.where(fine, s, 1.0)[..., None], 0.0)
    q = np.clip(np.rint(t), -qmax, qmax).astype(np.int64)
    return q, np.where(np.isfinite(s), s, np.nan), t


def unpack(codes, bits: int):
    """Stored bytes -> q, along the last axis."""
    c = np.asarray(codes).astype(np.int64)
    if bits == 4:
        c = np.stack([c & 15, c >> 4], axis=-1).reshape(*c.shape[:-1], -1)
    return c - 2 ** (bits - 1)


def pack(q, bits: int):
    u = (np.asarray(q) + 2 ** (bits - 1)).astype(np.uint8)
    return u if bits == 8 else (u[..., 0::2] | (u[..., 1::2] << 4)).astype(np.uint8)


def held(codes, scales, table, s: int, positions, head: int, bits: int):
    """Rotated vectors of sequence s at the positions, and which of them exist."""
    pages, _, page_size, _ = codes.shape
    d = codes.shape[3] * 8 // bits
    out, there = np.zeros((len(positions), d)), np.zeros(len(positions), dtype=bool)
    for i, p in enumerate(positions):
        at = slot(table, pages, page_size, s, int(p))
        if at is None:
            continue
        there[i] = True
        out[i] = unpack(codes[at[0], head, at[1]], bits) * np.float64(scales[at[0], head, at[1]])
    return out, there


def visible(pos: int, length: int, causal: bool, window: int):
    """Positions a token at pos sees."""
    hi = min(length, pos + 1) if causal else length
    lo = max(0, pos - window + 1) if window else 0
    return range(lo, hi)


def attention(q, k, v, table, cu, lens, bits, k_signs, v_signs, scale, causal=True, window=0, inv_freq=None,
              interleaved=False, positions=None, axis=None):
    """out [tokens, heads, d] (0 where nothing is seen, NaN rows for tokens of no sequence), and for every
    output vector the pair (largest sum_i |q_i k_i| * |scale|, sum_j p_j |v_j|) its error bounds are made of.
    k, v: (codes, scales)."""
    tokens, heads, d = q.shape
    hk = k[0].shape[1]
    out = np.full((tokens, heads, d), np.nan)
    size = np.zeros((tokens, heads, 2))
    for s in range(len(lens)):
        mine = [(t, p) for t, (o, p) in enumerate(places(cu, lens, tokens)) if o == s]
        length = int(lens[s])
        for h in range(hk):
            if not mine:
                continue
            kk, there = held(k[0], k[1], table, s, range(length), h, bits)
            vv, _ = held(v[0], v[1], table, s, range(length), h, bits)
            for t, p in mine:
                see = np.array([j for j in visible(p, length, causal, window) if there[j]], dtype=int)
                for g in range(heads // hk):
                    hq = h * (heads // hk) + g
                    x = np.asarray(q[t, hq], dtype=np.float64)
                    if inv_freq is not None:
                        x = rope(x, angles(inv_freq, p, t, positions, axis), interleaved)
                    x = rotate(x, k_signs)
                    if len(see) == 0:
                        out[t, hq] = 0.0
                        continue
                    z = kk[see] @ x * scale
                    w = np.exp(z - z.max())
                    w /= w.sum()
                    out[t, hq] = unrotate(w @ vv[see], v_signs)
                    size[t, hq] = (np.abs(kk[see]) @ np.abs(x)).max() * abs(scale), w @ np.linalg.norm(vv[see], axis=1)
    return out, size
