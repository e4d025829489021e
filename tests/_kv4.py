"""Plain 64-bit forms of the softmax-attention layers' operators, and the 4-bit cache's format byte by byte
(numpy; shares nothing with the library)."""
from __future__ import annotations

import numpy as np

GROUP = 32


def bf16_bits(x):
    """Bits of the bf16 nearest to fp32 values (ties to even); NaN -> 0x7fc0."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint32)
    return np.where(np.isnan(np.asarray(x, np.float32)), 0x7FC0, r).astype(np.uint16)


def bf16_values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def quantise(x):
    """x [..., D] -> codes int [..., D], scales fp64 [..., D/32] (NaN for a group that is not finite)."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        m = np.max(np.abs(g), axis=-1)
        fine = np.isfinite(m)
        m = np.where(fine, m, 1.0) / 7.0
        e = np.floor(np.log2(np.where(m > 0, m, 1.0))) - 4
        s = np.clip(np.ceil(m / 2.0 ** e) * 2.0 ** e, 2.0 ** -100, 2.0 ** 123)
        c = np.clip(np.round(np.where(fine[..., None], g, 0.0) / s[..., None]), -7, 7).astype(int) + 8
    return c.reshape(x.shape), np.where(fine, s, np.nan)


def held(x):
    """What a cache that was given x holds."""
    c, s = quantise(x)
    return (c - 8) * np.repeat(s, GROUP, axis=-1)


def empty_cache(pages, Hk, page, D, fill=0):
    return np.full((pages, Hk, page // 16, 18 * D), fill, dtype=np.uint8)


def _places(D, t, ch):
    """(byte of the half, bit in it) of a token's key and value channel in its block, and of its group's scales."""
    G, g, w, odd, nib = D // 32, ch // 32, ch % 32 // 8, ch % 2, ch % 8 // 2
    r, p = 2 * w + odd, t // 2
    key = t * (D // 2) + w * (D // 8) + 4 * g + 2 * odd
    value = 9 * D + p * D + ((r + 2 * p) % 8) * (D // 8) + (t % 2) * 2 * G + 2 * g
    return key, value, nib, 8 * D + t * 2 * G + 2 * g, 17 * D + p * 4 * G + 4 * g + 2 * (t % 2)


def put(block, t, k, v):
    """Write a token's keys and values [D] into its block (uint8 [18 D]) as token t of 16."""
    D = k.shape[0]
    for which, x in ((0, k), (1, v)):
        codes, s = quantise(x)
        for ch in range(0, D, 8):
            for odd in range(2):
                h = 0
                for i in range(4):
                    h |= int(codes[ch + odd + 2 * i]) << (4 * i)
                h = ((h << 3) | (h >> 13)) & 0xFFFF
                at = _places(D, t, ch + odd)[which]
                block[at], block[at + 1] = h & 255, h >> 8
        for g in range(D // 32):
            at = _places(D, t, 32 * g)[3 + which]
            b = int(bf16_bits(s[g:g + 1])[0])
            block[at], block[at + 1] = b & 255, b >> 8


def get(block, t, D):
    """The inverse of put: keys and values [D] in fp64."""
    out = []
    for which in range(2):
        x = np.empty(D)
        for ch in range(D):
            at = _places(D, t, ch)
            h = int(block[at[which]]) | int(block[at[which] + 1]) << 8
            h = ((h >> 3) | (h << 13)) & 0xFFFF
            code = (h >> (4 * at[2])) & 15
            s = int(block[at[3 + which]]) | int(block[at[3 + which] + 1]) << 8
            x[ch] = (code - 8) * bf16_values(s)
        out.append(x)
    return out


def tokens(cache, table, b, n):
    """Keys and values [n, Hk, D] of the first n tokens of sequence b."""
    Hk, page, D = cache.shape[1], cache.shape[2] * 16, cache.shape[3] // 18
    ch = np.arange(D)
    k, v = np.empty((n, Hk, D)), np.empty((n, Hk, D))
    for i in range(n):
        blk = cache[table[b, i // page], :, i % page // 16].astype(np.int64)  # [Hk, 18 D]
        key, value, nib, ks, vs = _places(D, i % 16, ch)
        for at, sc, x in ((key, ks, k), (value, vs, v)):
            h = blk[:, at] | blk[:, at + 1] << 8
            h = ((h >> 3) | (h << 13)) & 0xFFFF
            x[i] = ((h >> (4 * nib)) & 15) - 8
            x[i] *= bf16_values(blk[:, sc] | blk[:, sc + 1] << 8)
    return k, v


def attention(q, k, v, pos, scale, causal, window):
    """q [n, Hq, D] at positions pos [n] over k, v [L, Hk, D]. Returns out, lse, the largest size of the terms
    of each output (sum p |v|) and of each row's scores (max over tokens of scale * sum |q k|)."""
    n, Hq, D = q.shape
    L, Hk = k.shape[:2]
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    terms, size = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    j = np.arange(L)
    for h in range(Hq):
        g = h // (Hq // Hk)
        for i in range(n):
            see = (j <= pos[i]) if causal else np.ones(L, bool)
            if window:
                see &= j > pos[i] - window
            if not see.any():
                continue
            s = scale * (k[see, g] @ q[i, h])
            size[i, h] = scale * np.max(np.abs(k[see, g]) @ np.abs(q[i, h]))
            m = np.max(s)
            p = np.exp(s - m)
            lse[i, h] = m + np.log(p.sum())
            out[i, h] = p @ v[see, g] / p.sum()
            terms[i, h] = p @ np.abs(v[see, g]) / p.sum()
    return out, lse, terms, size


def norm_rope(x, w, pos, freq, eps, interleaved):
    """x [T, H, D]; w [D] or None; pos int [T], freq fp64 [R/2] or None."""
    y = np.asarray(x, np.float64).copy()
    if w is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    if freq is not None and len(freq):
        # turns modulo one in exact integers: 2^64 units to a turn
        unit = [int(round((float(f) / (2 * np.pi) % 1.0) * 2 ** 64)) for f in freq]
        turn = np.array([[(int(p) * u % 2 ** 64) / 2.0 ** 64 for u in unit] for p in pos]) * 2 * np.pi
        c, s = np.cos(turn)[:, None], np.sin(turn)[:, None]
        n = len(freq)
        a, b = (y[..., 0:2 * n:2], y[..., 1:2 * n:2]) if interleaved else (y[..., :n], y[..., n:2 * n])
        a, b = a * c - b * s, b * c + a * s
        if interleaved:
            y[..., 0:2 * n:2], y[..., 1:2 * n:2] = a, b
        else:
            y[..., :n], y[..., n:2 * n] = a, b
    return y
