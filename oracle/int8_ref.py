"""Oracle of the RMS norm, its gradient, the row-scaled 8-bit integer codes and
the int8 2:4 product.  TEST INFRASTRUCTURE ONLY; shares no code with the library.

Arrays are float64 holding exactly widened stored values (or int codes);
results are float64 and unrounded unless the step itself rounds.
"""
from __future__ import annotations

import numpy as np

from .slope_ref import decompress24, round_bf16, round_f16, round_f32

__all__ = ["residual_sum", "rmsnorm", "rmsnorm_bwd", "row_codes_i8", "spmm_i8", "round_to"]


def round_to(x, fmt: str) -> np.ndarray:
    """Nearest value of the format ("bf16", "f16" or "f32"), as float64."""
    x = np.asarray(x, np.float64)
    out = {"bf16": round_bf16, "f16": round_f16, "f32": round_f32}[fmt](x)
    if fmt == "bf16":
        return (np.asarray(out).astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)
    return out.astype(np.float64)


def residual_sum(x, res, fmt: str) -> np.ndarray:
    """h = x + res, the float32 sum rounded to the storage format."""
    if res is None:
        return np.asarray(x, np.float64)
    return round_to((x.astype(np.float32) + res.astype(np.float32)).astype(np.float64), fmt)


def rmsnorm(h, gamma, eps):
    """(y, rstd) of h [T, K]."""
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    y = h * rstd[:, None]
    return (y if gamma is None else y * gamma), rstd


def rmsnorm_bwd(dy, h, rstd, gamma, dh=None):
    """(dX, dgamma) given the forward's rstd [T]."""
    xh = h * rstd[:, None]
    a = dy if gamma is None else dy * gamma
    dx = rstd[:, None] * (a - xh * (a * xh).mean(axis=1, keepdims=True))
    return (dx if dh is None else dx + dh), (dy * xh).sum(axis=0)


def row_codes_i8(u):
    """(codes int8 [R, K], amax [R]) of rows u: the integer nearest to 127 u /
    amax, ties to even; rows with an infinity or a NaN get codes 0 and amax NaN.

    In float64 127 u is exact for products of two 16-bit values or of a 16-bit
    and a float32 value (at most 42 bits), and the one division is correctly
    rounded, so a quotient that is a tie stays one.  Any other quotient q >= 1/2
    differs from a tie by |254 u - (2k + 1) amax| / (2 amax), whose numerator is
    a multiple of u's last place (2^-35 u at least): far more than 2^-46, half
    of float64's spacing below 128."""
    u = np.asarray(u, np.float64)
    amax = np.abs(u).max(axis=1) if u.shape[1] else np.zeros(u.shape[0])
    bad = ~np.isfinite(u).all(axis=1)
    safe = np.where(bad | (amax == 0), 1.0, amax)
    q = np.rint(127.0 * np.where(bad[:, None], 0.0, u) / safe[:, None])
    return q.astype(np.int8), np.where(bad, np.nan, amax)


def spmm_i8(xq, x_scale, wq_values, meta, K, w_scale, fmt: str):
    """Y [T, N]: the exact integer product, converted to float32, times the
    float32 product of the scales, rounded to the format."""
    w = decompress24(wq_values, meta, K).astype(np.float64)
    acc = xq.astype(np.float64) @ w.T                # integers below 2^53: exact
    s = x_scale.astype(np.float32)[:, None] * w_scale.astype(np.float32)[None, :]
    return round_to((acc.astype(np.float32) * s).astype(np.float64), fmt)
