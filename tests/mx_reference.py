"""Plain 64-bit implementations of MXFP4 and of the mixture-of-experts layer, from their definitions.

Nothing here calls the library.  MXFP4 codes are decoded from their bits and
chosen by comparison with the midpoints of neighbouring values; sums are NumPy
float64.  `bound` arguments: every product returns (y, e), e an elementwise
limit on the error of the library's fp32 arithmetic, from these counts:

  * a BF16 rounding is within 2^-8 of its value (half a unit of the last of 8 bits);
  * an fp32 sum of n exact products is within n 2^-23 of the sum of their
    magnitudes (n roundings of at most 2^-24 each, doubled for adders that cut off);
  * exp, the reciprocal and the division in the softmax and in silu are within
    2^-18 of their values for the arguments used (a few units of 2^-23, and the
    argument's own rounding times up to 16).
"""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """float32 -> BF16 bit patterns, round to nearest even (finite values)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_values(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def decode_codes(codes: np.ndarray) -> np.ndarray:
    """uint8 [..., K/2] -> float64 [..., K]: sign bit 3, exponent bits 2..1, mantissa bit 0."""
    q = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).astype(np.int64)
    e, m, s = (q >> 1) & 3, q & 1, q >> 3
    return np.where(s == 1, -1.0, 1.0) * np.where(e == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (e - 1))


def decode(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """MXFP4 -> float64; a block with scale byte 255 is NaN."""
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return decode_codes(codes) * np.repeat(s, 32, axis=-1)


def encode(x: np.ndarray):
    """float64/float32 [R, K] -> (codes uint8 [R, K/2], scales uint8 [R, K/32])."""
    R, K = x.shape
    v = x.astype(np.float64).reshape(R, K // 32, 32)
    bad = ~np.isfinite(v).all(-1)
    a = np.where(bad, 0.0, np.abs(np.where(np.isfinite(v), v, 0.0)).max(-1))
    _, ex = np.frexp(a)  # a = f 2^ex, f in [0.5, 1): floor(log2 a) = ex - 1
    s = np.where(a > 0, np.maximum(ex - 1 - 2 + 127, 0), 0)
    s = np.where(a < 2.0 ** -126, 0, s)
    z = np.where(np.isfinite(v), v, 0.0) / (2.0 ** (s.astype(np.float64) - 127))[..., None]
    mag = np.abs(z)
    q = np.zeros(mag.shape, np.int64)
    for c in range(1, 8):  # the midpoint itself goes to the even one of the two codes
        mid = (MAGNITUDES[c - 1] + MAGNITUDES[c]) / 2
        q = np.where((mag > mid) | ((mag == mid) & (c % 2 == 0)), c, q)
    q = q + 8 * np.signbit(z)
    q = np.where(bad[..., None], 0, q).reshape(R, K)
    codes = (q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8)
    return codes, np.where(bad, 255, s).astype(np.uint8)


def product(x: np.ndarray, w: np.ndarray):
    """y = x w^T with its error limit; float64 [m, K], [N, K]."""
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    return y, 2.0 ** -8 * np.abs(y) + x.shape[1] * 2.0 ** -23 * mag


def affine_weight(codes: np.ndarray, scales_bits: np.ndarray, biases_bits: np.ndarray, gs: int):
    """8-bit affine weight and the magnitudes of its two terms, float64 [N, K]."""
    s = np.repeat(bf16_values(scales_bits), gs, axis=1)
    b = np.repeat(bf16_values(biases_bits), gs, axis=1)
    q = codes.astype(np.float64)
    return q * s + b, q * np.abs(s) + np.abs(b)


def route(logits: np.ndarray, topk: int, renorm: bool, scale: float):
    """float64 [T, E] -> weights [T, E] (0: not taken); NaN rows where the logits hold NaN or +inf."""
    T, E = logits.shape
    r = np.zeros((T, E))
    for t in range(T):
        l = logits[t]
        if np.isnan(l).any() or (l == np.inf).any():
            r[t] = np.nan
            continue
        if (l == -np.inf).all():
            continue
        p = np.exp(l - l.max())
        order = sorted(range(E), key=lambda j: (-l[j], j))[:topk]
        order = [j for j in order if l[j] > -np.inf]
        total = p[order].sum() if renorm else p.sum()
        r[t, order] = scale * p[order] / total
    return r


def moe(x, gate, up, down, mags, logits, topk, renorm=True, scale=1.0, resid=None):
    """The layer in float64: (y, limit).  gate, up [E, I, H], down [E, H, I]; mags: the magnitudes behind their sums."""
    r = route(logits, topk, renorm, scale)
    T, H = x.shape
    E, I = gate.shape[:2]
    y = np.zeros((T, H)) if resid is None else resid.copy()
    err = np.zeros((T, H))
    for e in range(E):
        on = np.flatnonzero(r[:, e] > 0) if scale > 0 else np.flatnonzero(r[:, e] < 0)
        if on.size == 0:
            continue
        xe = x[on]
        g, u = xe @ gate[e].T, xe @ up[e].T
        dg = H * 2.0 ** -23 * (np.abs(xe) @ mags[0][e].T)
        du = H * 2.0 ** -23 * (np.abs(xe) @ mags[1][e].T)
        with np.errstate(over="ignore"):
            s = g / (1 + np.exp(-g))
        w = r[on, e][:, None]
        h = w * s * u
        # |silu'| <= 1.1; the rounding of h to BF16 and of its factors
        dh = np.abs(w) * (1.1 * dg * (np.abs(u) + du) + np.abs(s) * du) + (2.0 ** -8 + 2.0 ** -16) * np.abs(h)
        y[on] += h @ down[e].T
        err[on] += dh @ np.abs(down[e]).T + I * 2.0 ** -23 * ((np.abs(h) + dh) @ mags[2][e].T)
    nan = np.isnan(r).any(1)
    y[nan] = np.nan
    return y, err + (topk + 2) * 2.0 ** -23 * np.abs(y) + 2.0 ** -8 * (np.abs(y) + err)
