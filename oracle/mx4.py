"""MXFP4 rows and products with both operands in MXFP4, float64.

The format is oracle/mxfp4.py's; quantisation follows the OCP MX v1.0 element
definition (round to nearest, ties to even mantissa, saturating) with one of
two scale rules:
  fit  the smallest power of two with amax <= 6 * scale
  ocp  2**(floor(log2(amax)) - 2)
scale exponents held to [-125, 126] (a block of zeros takes -125); a block with
a value that is not finite takes the scale byte 255 and codes of zero.
"""
from __future__ import annotations

import numpy as np

from .layer import situ_glu
from .mxfp4 import E2M1_VALUES, GROUP, e8m0_to_f64, unpack_codes


def scale_exponent(amax: np.ndarray, rule: str) -> np.ndarray:
    """Exponent of the block scale for finite amax >= 0."""
    if rule not in ("fit", "ocp"):
        raise ValueError(rule)
    m, p = np.frexp(np.asarray(amax, np.float64))  # amax = m 2^p, m in [0.5, 1); 6 = 0.75 2^3
    e = p - 3
    if rule == "fit":
        e = np.where(m > 0.75, e + 1, e)
    return np.clip(np.where(m == 0, -125, e), -125, 126)


def grid(t: np.ndarray) -> np.ndarray:
    """t on the e2m1 grid: nearest, ties to even mantissa, at most 6."""
    a = np.abs(t)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    return np.copysign(np.minimum(np.round(a / step) * step, 6.0), t)


def quantize(x: np.ndarray, rule: str = "fit"):
    """(packed codes u8 [T, ceil(K / 2)], scale bytes u8 [T, ceil(K / 32)]) of x [T, K]."""
    T, K = x.shape
    kb = -(-K // GROUP)
    b = np.zeros((T, kb * GROUP))
    b[:, :K] = x
    b = b.reshape(T, kb, GROUP)
    bad = ~np.isfinite(b).all(2)
    b = np.where(bad[:, :, None], 0.0, b)
    e = scale_exponent(np.abs(b).max(2), rule)
    v = grid(np.ldexp(b, -e[:, :, None]))
    mag = np.searchsorted(E2M1_VALUES[:8], np.abs(v)).astype(np.uint8)
    code = np.where(bad[:, :, None], 0, mag | (np.signbit(v).astype(np.uint8) << 3)).reshape(T, -1).astype(np.uint8)
    code = code[:, :2 * (-(-K // 2))]
    return code[:, 0::2] | (code[:, 1::2] << 4), np.where(bad, 255, e + 127).astype(np.uint8)


def dequantize(q: np.ndarray, s: np.ndarray, K: int) -> np.ndarray:
    """Values [..., K] of packed codes [..., ceil(K / 2)] and scale bytes [..., ceil(K / 32)]."""
    return E2M1_VALUES[unpack_codes(q)][..., :K] * np.repeat(e8m0_to_f64(s), GROUP, axis=-1)[..., :K]


def expert_product(x, w, offsets, w3=None, rows=None, pair_weight=None, beta=4.0, beta_lin=25.0):
    """Rows p of expert e: x[rows[p]] w[e]^T, times pair_weight[p], or SiTU-GLU of that and x[rows[p]] w3[e]^T.
    All values already dequantised; rows past offsets[-1] are NaN.  Returns (result, gate product, sum of magnitudes)."""
    P = len(rows)
    out, gate, mag = (np.full((P, w.shape[1]), np.nan) for _ in range(3))
    for e in range(w.shape[0]):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        a = x[rows[s]]
        gate[s] = a @ w[e].T
        mag[s] = np.abs(a) @ np.abs(w[e]).T
        out[s] = gate[s] if w3 is None else situ_glu(gate[s], a @ w3[e].T, beta, beta_lin)
        if pair_weight is not None:
            out[s] *= pair_weight[s, None]
    return out, gate, mag
