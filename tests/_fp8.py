"""fp64 statements of the 8-bit operators and the tolerances their tests use.

Tolerances are sums of rounding errors, counted before any run:
  U = 2^-24 is half a step of fp32 relative to the value.
"""
from __future__ import annotations

import numpy as np

BLOCK, QMAX, AMAX_MIN = 128, 448.0, 2.0 ** -96
U = 2.0 ** -24


def _e4m3_table():
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = np.nan if e == 15 and m == 7 else (m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[c] = -x if c & 128 else x
    return v


E4M3 = _e4m3_table()


def codes_to_np(t):
    """float8_e4m3fn tensor -> the values of its codes in fp64."""
    import torch
    return E4M3[t.contiguous().view(torch.uint8).cpu().numpy()]


def nblocks(n):
    return -(-n // BLOCK)


def per_channel(s, n):
    """Scales [blocks, T] -> [T, n], one per channel."""
    return np.repeat(np.asarray(s, np.float64).T, BLOCK, axis=1)[:, :n]


def block_scales(y):
    """[T, n] fp64 -> scales [blocks, T]; NaN is ignored by the maximum."""
    t, n = y.shape
    out = np.empty((nblocks(n), t))
    for b in range(out.shape[0]):
        a = np.abs(y[:, b * BLOCK:(b + 1) * BLOCK])
        out[b] = np.maximum(np.max(np.where(np.isnan(a), 0.0, a), axis=1), AMAX_MIN) / QMAX
    return out


def add_rmsnorm(x, residual, w, eps):
    h = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    den = (h * h).mean(-1, keepdims=True) + eps
    inv = np.where(den > 0, 1 / np.sqrt(np.where(den > 0, den, 1)), 0.0)
    return h, h * inv * np.asarray(w, np.float64)


def check_codes(y, codes, scales, steps, what=""):
    """codes (fp64 values) and scales [blocks, T] of finite y [T, n], computed in fp32 with at most
    `steps` half-steps of relative error in each y. The scale carries that error and its division
    (2 more); a code is the value's, with that error, its scale's, the reciprocal's and the product's
    (3 more), and half a step of e4m3: 2^-4 of the value, or 2^-10 below the smallest normal 2^-6."""
    s = np.asarray(scales, np.float64)
    ref = block_scales(y)
    rel = np.max(np.abs(s - ref) / ref) if ref.size else 0.0
    assert rel <= (steps + 2) * U, f"{what}: scale off by {rel:.3e}, {rel / U:.1f} half-steps of {steps + 2}"
    v = y / per_channel(s, y.shape[1])
    err = np.abs(codes - v)
    tol = np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) + np.abs(v) * (2 * steps + 5) * U
    assert np.all(np.isfinite(codes)), f"{what}: non-finite codes"
    assert np.all(err <= tol), f"{what}: code off by {np.max(err / np.maximum(tol, 1e-300)):.3f} of its bound"


def add_norm_steps(n):
    """Half-steps of fp32 that y of kda_add_rmsnorm_fp8 may be off by. Each channel's square passes at
    most 8 * 4 (a thread's channels) + 5 + 5 (two shuffle trees) roundings on its way into the sum, twice
    that for the fp32 sum h itself (its square doubles the error); the square root halves them, the mean
    and eps, root and reciprocal add 4, the two products 2 and h 1."""
    return (8 * 4 + 10 + 2) / 2 + 4 + 2 + 1


def gated_steps(zmax):
    """The same for kda_gated_rmsnorm_fp8: 8 + 4 roundings in the sum of squares, halved, 4 for mean, root
    and reciprocal, 4 products; exp(-z) as 2^(z log2 e): the argument's rounding is |z| half-steps of the
    result (log2 e times ln 2 is 1), its own rounding 1, the hardware exponential 4, the sum 1, the fast
    division 4."""
    return 6 + 4 + 4 + abs(zmax) + 1 + 4 + 1 + 4


def linear(a, sa, w, sw):
    """a [M,K], w [N,K] code values; sa [KB,M], sw [NB,KB]. Returns (y, sum of magnitudes)."""
    K, N = a.shape[1], w.shape[0]
    y = np.zeros((a.shape[0], N))
    mag = np.zeros_like(y)
    rows = np.arange(N) // BLOCK
    sw, sa = np.asarray(sw, np.float64), np.asarray(sa, np.float64)
    for b in range(nblocks(K)):
        c = slice(b * BLOCK, (b + 1) * BLOCK)
        s = sa[b][:, None] * sw[rows, b][None, :]
        y += (a[:, c] @ w[:, c].T) * s
        mag += (np.abs(a[:, c]) @ np.abs(w[:, c]).T) * np.abs(s)
    return y, mag


def check_linear(got, a, sa, w, sw, bf16, what=""):
    """Each addition on the tensor cores may cut instead of round: a whole step (2 half-steps) of at most
    the magnitudes' sum, for 128 products of a block; the scale's product, its multiply-add and the nkb
    additions of the blocks round: 2 + nkb half-steps; a bf16 result rounds by 2^-8 of its value."""
    y, mag = linear(a, sa, w, sw)
    nkb = nblocks(a.shape[1])
    tol = mag * (2 * 128 + 2 + nkb) * U + (np.abs(y) * 2.0 ** -8 if bf16 else 0.0) + 1e-37
    got = np.asarray(got, np.float64)
    assert np.all(np.isfinite(got)), f"{what}: non-finite result"
    err = np.abs(got - y)
    assert np.all(err <= tol), f"{what}: off by {np.max(err / tol):.3f} of its bound"
