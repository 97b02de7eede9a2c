"""ORACLE (test infrastructure only): 8-bit floating point with block scales, float64.

e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; exponent 0 holds the subnormals m * 2^-9; the
code with all exponent and mantissa bits set is NaN; there is no infinity, the largest value is 448.

Rows are quantised in groups of 128 columns (the last may be shorter): m the largest magnitude,
s = max(fl32(m / 448), 2^-126), q = e4m3(fl32(v * fl32(1 / s))), ties to even.  Matrices carry one
scale per 128 x 128 block.
"""
import numpy as np


def decode(bits: np.ndarray) -> np.ndarray:
    """e4m3 bit patterns (uint8) -> float64."""
    b = np.asarray(bits, dtype=np.uint8).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, np.ldexp(m.astype(np.float64), -9), np.ldexp(8.0 + m, e - 10))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >> 7 == 1, -v, v)


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """float64 values of magnitude below 464 -> the nearest e4m3 value (float64), ties to even; NaN stays."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(np.where(np.isfinite(v), v, 0.0))
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(v / step) * step


def quantise(rows: np.ndarray):
    """float64 rows [T, d] -> (q values float64 [T, d], scales float64 [T, ceil(d/128)])."""
    rows = np.asarray(rows, dtype=np.float64)
    q = np.empty_like(rows)
    scales = []
    with np.errstate(invalid="ignore", over="ignore"):
        for c in range(0, rows.shape[1], 128):
            g = rows[:, c:c + 128]
            s = (np.abs(g).max(axis=1) / 448.0).astype(np.float32)
            s = np.where(s < np.float32(2.0 ** -126), np.float32(2.0 ** -126), s)
            r = (1.0 / s.astype(np.float64)).astype(np.float32).astype(np.float64)
            q[:, c:c + 128] = round_e4m3((g * r[:, None]).astype(np.float32).astype(np.float64))
            scales.append(s.astype(np.float64))
    return q, np.stack(scales, axis=1)


def rows_value(q: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The values that quantised rows stand for."""
    return q * np.repeat(scales, 128, axis=1)[:, :q.shape[1]]


def matrix_value(bits: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """e4m3 bit patterns [R, K] with a scale per 128 x 128 block -> float64 [R, K]."""
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), 128, axis=0), 128, axis=1)
    return decode(bits) * s[:bits.shape[0], :bits.shape[1]]


def swiglu_expert_fp8(a, wg, wu, wd):
    """SwiGLU of quantised rows: a [n, d] and h are quantised before their products; wg, wu, wd the
    matrices' values (matrix_value)."""
    a = rows_value(*quantise(a))
    g, u = a @ wg.T, a @ wu.T
    h = (g / (1.0 + np.exp(-g))) * u
    return rows_value(*quantise(h)) @ wd.T


def add_rmsnorm(x, residual, weight, eps, round_sum):
    """-> (h, y) float64; round_sum rounds the sum to the rows' type."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = round_sum(h + np.asarray(residual, np.float64))
    return h, h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)
