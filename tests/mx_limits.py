"""Statistical limits for the MXFP4 products and the expert layer, beside the worst case of mx_reference.py.

The worst case adds the magnitudes of all roundings, which grows with the length of a row until a lost block
fits in.  Roundings have no common sign, so what they add up to is much less:

  * the output's rounding to BF16 is within 2^-8 of each value, so within 2^-8 of a row in L2 too;
  * K additions in fp32 of terms of no common sign: each rounds by up to 2^-24 of a partial sum, which is about
    the row's rms, together sqrt(K) 2^-24 rms; eight times that is allowed;
  * the layer keeps h in BF16: an rms error of at most 2^-9 of each h, independent of each other, so a normal
    error of 2^-9 of the row's rms in y; six sigmas are allowed to an element.  In L2 the two roundings make
    0.0024 of a row; twice that is allowed.

They hold for rows whose terms have random signs and comparable sizes, which the inputs made here have: scales
within a factor of 32, and routing weights of the same order.  Nothing here calls the library.
"""
from __future__ import annotations

import numpy as np

import mx_reference as R


def rms(ref: np.ndarray) -> np.ndarray:
    return np.sqrt(np.mean(ref * ref, axis=1, keepdims=True))


def product_faults(y: np.ndarray, ref: np.ndarray, K: int) -> list[str]:
    """What is beyond the limits of a product with rows of K; empty: nothing."""
    return _faults(y, ref, K ** 0.5 * 2.0 ** -21, 2.0 ** -8 + K ** 0.5 * 2.0 ** -21)


def layer_faults(y: np.ndarray, ref: np.ndarray, inner: int, hidden: int) -> list[str]:
    fp32 = (inner ** 0.5 + 3 * hidden ** 0.5) * 2.0 ** -21  # the down sum, and gate and up twice for silu's slope
    return _faults(y, ref, 6 * 2.0 ** -9 + fp32, 0.005 + fp32)


def _faults(y, ref, of_rms, of_norm):
    d = np.abs(y - ref)
    bad = ~(d <= 2.0 ** -8 * np.abs(ref) + of_rms * rms(ref))  # NaN is beyond it too
    rows = np.sqrt(np.sum(d * d, axis=1) / np.sum(ref * ref, axis=1))
    out = []
    if bad.any():
        out.append(f"{np.count_nonzero(bad)} of {bad.size} elements, first {np.argwhere(bad)[0]}: "
                   f"got {y[bad][0]}, want {ref[bad][0]}")
    if not (rows <= of_norm).all():
        out.append(f"relative L2 error of row {int(np.argmax(rows))} is {rows.max():.5f}, limit {of_norm:.5f}")
    return out


def rounded(x: np.ndarray) -> np.ndarray:
    return R.bf16_values(R.bf16_bits(np.asarray(x, np.float32)))


def mx_matrix(seed: int, rows: int, k: int):
    """Codes, and scales within a factor of 32."""
    rng = np.random.default_rng(seed)
    return rng.integers(0, 256, (rows, k // 2), np.uint8), rng.integers(117, 122, (rows, k // 32), np.uint8)


class Experts:
    """A layer's weights as raw arrays: raw[i] of gate, up, down, [E * rows, k]; scales differ from group to group."""

    def __init__(self, seed: int, fmt: str, E: int, I: int, H: int):
        self.fmt, self.E, self.I, self.H = fmt, E, I, H
        self.gs = 32 if fmt == "mxfp4" else int(fmt[2:])
        self.raw = []
        for i, (n, k) in enumerate(((E * I, H), (E * I, H), (E * H, I))):
            if fmt == "mxfp4":
                self.raw.append(list(mx_matrix(seed + i, n, k)))
            else:
                rng = np.random.default_rng(seed + i)
                s = R.bf16_bits(rng.uniform(1e-4, 4e-4, (n, k // self.gs)).astype(np.float32))
                b = -128 * R.bf16_values(s) * (1 + rng.uniform(-0.05, 0.05, s.shape))
                self.raw.append([rng.integers(0, 256, (n, k), np.uint8), s, R.bf16_bits(b.astype(np.float32))])

    def values(self, i: int) -> np.ndarray:
        """float64 [E, rows, k]."""
        w = R.decode(*self.raw[i]) if self.fmt == "mxfp4" else R.affine_weight(*self.raw[i], self.gs)[0]
        return w.reshape(self.E, -1, w.shape[1])

    def upload(self):
        import torch
        from weight_only_quantized_int8_amd import Int8Weight, Mxfp4Weight
        if self.fmt == "mxfp4":
            return [Mxfp4Weight(*(torch.from_numpy(a).cuda() for a in r)) for r in self.raw]
        return [Int8Weight.from_arrays(c.view(np.uint32), s, b, self.gs) for c, s, b in self.raw]


def layer(x, W, logits, topk, round_h=False):
    """The layer in float64, renormalized; round_h: with h in BF16, as the kernels keep it."""
    r = R.route(logits, topk, True, 1.0)
    y = np.zeros((x.shape[0], W[2].shape[1]))
    for e in range(logits.shape[1]):
        on = np.flatnonzero(r[:, e] > 0)
        if on.size:
            g, u = x[on] @ W[0][e].T, x[on] @ W[1][e].T
            h = r[on, e][:, None] * g / (1 + np.exp(-g)) * u
            y[on] += (rounded(h) if round_h else h) @ W[2][e].T
    return y


def layer_inputs(seed: int, T: int, H: int, E: int):
    """x in BF16 bits, and logits whose chosen experts get weights of the same order."""
    rng = np.random.default_rng(seed)
    return R.bf16_bits(rng.standard_normal((T, H)).astype(np.float32)), (0.3 * rng.standard_normal((T, E))).astype(np.float32)
