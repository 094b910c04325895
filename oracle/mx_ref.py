"""Oracle of the microscaled formats: AdamW with 8-bit moments and 4-bit floating
point with its product.  TEST INFRASTRUCTURE ONLY; shares no code with the library.

A scale is one byte b for a block of 32 values, 2^(b - 127), 255 = NaN.  Codes are
enumerated: a format is the table of its codes' magnitudes.
"""
from __future__ import annotations

import numpy as np

__all__ = ["MX_BLOCK", "float_grid", "moments8", "moment_codes8", "random_words", "tensor_seed", "adamw_f32",
           "adamw8"]

MX_BLOCK = 32
TOP_M, TOP_V = 7, 15


def float_grid(exp_bits: int, mant_bits: int, bias: int) -> np.ndarray:
    """Magnitudes of all codes of a small float format without special values."""
    out = []
    for e in range(1 << exp_bits):
        for f in range(1 << mant_bits):
            frac = f / (1 << mant_bits)
            out.append(2.0 ** (1 - bias) * frac if e == 0 else 2.0 ** (e - bias) * (1 + frac))
    return np.array(out)


GRID_M = float_grid(4, 3, 7)       # E4M3's magnitudes (the last one is its NaN: never written)
GRID_V = float_grid(5, 3, 15)


def _scales(exps, n):
    s = np.ldexp(1.0, exps.astype(np.int64) - 127)
    s = np.where(exps == 255, np.nan, s)
    return np.repeat(s, MX_BLOCK)[:n]


def moments8(m, m_exp, v, v_exp):
    """(m, v) in float64 from codes [n] and scales [ceil(n / 32)]."""
    n = m.size
    mv = np.where(m & 0x80, -1.0, 1.0) * np.where((m & 0x7F) == 0x7F, np.nan, GRID_M[m & 0x7F]) * _scales(m_exp, n)
    return mv, GRID_V[v] * _scales(v_exp, n)


def tensor_seed(seed: int, i: int) -> int:
    """The 32-bit seed of tensor i (SplitMix64)."""
    mask = (1 << 64) - 1
    z = (seed + (i + 1) * 0x9E3779B97F4A7C15) & mask
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
    return (z ^ (z >> 31)) & 0xFFFFFFFF


def random_words(n: int, seed32: int, first: int = 0) -> np.ndarray:
    """The 32-bit words of values first .. first + n - 1 (first a multiple of 8)."""
    runs = np.arange(first // 8, first // 8 + -(-n // 8)).astype(np.uint64)
    u = lambda x: x & np.uint64(0xFFFFFFFF)
    s = u(u(runs) * np.uint64(0x9E3779B1)) ^ np.uint64(seed32)
    s = u((s ^ (s >> np.uint64(16))) * np.uint64(0xBB67AE85))
    s ^= s >> np.uint64(15)
    out = np.empty((runs.size, 8), np.uint64)
    for j in range(8):
        s ^= u(s << np.uint64(13))
        s ^= s >> np.uint64(17)
        s ^= u(s << np.uint64(5))
        out[:, j] = s
    return out.reshape(-1)[:n]


def moment_codes8(x, noise20, grid, top, signed):
    """(codes, scales, values) of float32-valued moments x, rounded down after
    noise / 2^20 of a code's distance is added: position on the grid, counted in
    codes, linear between neighbours, to the nearest 2^-20 of a code."""
    n = x.size
    pad = np.zeros(-n % MX_BLOCK)
    blocks = np.concatenate([x, pad]).reshape(-1, MX_BLOCK)
    peak = np.abs(blocks).max(axis=1) if blocks.size else np.zeros(0)
    bad = ~np.isfinite(blocks).all(axis=1)
    e = np.where(bad | (peak == 0), 0, np.frexp(np.where(bad, 1.0, peak))[1] - 1)
    e = np.maximum(np.where(peak == 0, -127, e - top), -127)
    wide = np.repeat(e, MX_BLOCK)[:n]
    dead = np.repeat(bad, MX_BLOCK)[:n]
    a = np.where(dead, 0.0, np.ldexp(np.abs(np.where(dead, 0.0, x)), -wide))
    low = np.searchsorted(grid, a, side="right") - 1
    gap = grid[np.minimum(low + 1, grid.size - 1)] - grid[low]
    part = np.where(gap > 0, (a - grid[low]) / np.where(gap > 0, gap, 1.0), 0.0)
    code = low + (np.rint(part * 2 ** 20) + noise20 >= 2 ** 20)
    if not signed:
        code = np.maximum(code, a > 0)
    code = np.where(dead, 0, code).astype(np.uint8)
    if signed:
        code = np.where(dead, 0, code | (np.signbit(x).astype(np.uint8) << 7)).astype(np.uint8)
    exps = np.where(bad, 255, e + 127).astype(np.uint8)
    value = grid[code & 0x7F if signed else code] * _scales(exps, n) * (np.where(np.signbit(x), -1.0, 1.0) if signed else 1.0)
    return code, exps, value


def adamw_f32(g, m, v, beta1, beta2):
    """The new moments as the library's float32 operations give them, bit for bit:
    each product and each fused multiply-add rounds once.  (In long double a product
    of two float32 numbers is exact and a fused sum keeps 64 bits, so its one more
    rounding decides a float32 tie in one of 2^40 cases.)"""
    f = np.float32
    b1, o1, b2, o2 = f(beta1), f(1 - beta1), f(beta2), f(1 - beta2)
    L = np.longdouble
    with np.errstate(all="ignore"):
        g, m, v = (np.asarray(x).astype(f) for x in (g, m, v))
        gm = (o1 * g).astype(f)
        gv = (o2 * (g * g).astype(f)).astype(f)
        return ((L(b1) * m.astype(L) + gm.astype(L)).astype(f), (L(b2) * v.astype(L) + gv.astype(L)).astype(f))


def adamw8(g, m, m_exp, v, v_exp, beta1, beta2, seed32, first=0):
    """(m, m_exp, v, v_exp, m', v') of one step: the new codes and scales, and the
    moments before rounding (float32 numbers in float64)."""
    m0, v0 = moments8(m, m_exp, v, v_exp)
    mf, vf = (x.astype(np.float64) for x in adamw_f32(g, m0, v0, beta1, beta2))
    w = random_words(mf.size, seed32, first).astype(np.int64)
    cm, em, _ = moment_codes8(mf, w >> 12, GRID_M, TOP_M, True)
    cv, ev, _ = moment_codes8(vf, w & 0xFFFFF, GRID_V, TOP_V, False)
    return cm, em, cv, ev, mf, vf


# ------------------------------------------------------------------ 4-bit floating point

GRID4 = float_grid(2, 1, 1)        # E2M1's magnitudes

__all__ += ["mxfp4_codes", "mxfp4_values", "mxfp4_rows", "mxfp4_kept_codes", "spmm_mxfp4"]


def _block_codes(blocks):
    """(codes, scales) of rows that are one block each: the exponent is found by trying
    them, a code by the distance to every grid value."""
    R = blocks.shape[0]
    bad = ~np.isfinite(blocks).all(axis=1)
    x = np.where(bad[:, None], 0.0, blocks)
    peak = np.abs(x).max(axis=1) if x.size else np.zeros(R)
    # the largest E with peak >= 7 * 2^(E-1): from there on the peak rounds past 6 * 2^(E-1)
    e = np.full(R, -127)
    some = peak > 0
    guess = np.where(some, np.frexp(np.where(some, peak, 1.0))[1] - 4, -127)
    for _ in range(4):
        guess = np.where(some & (peak >= 7 * np.ldexp(1.0, guess)), guess + 1, guess)
    e = np.maximum(guess, -127)
    a = np.abs(x) * np.ldexp(1.0, -e)[:, None]
    d = np.abs(a[:, :, None] - GRID4)
    best = d.min(axis=2)
    low = np.argmin(d, axis=2)                       # of a tie the lower one; the even one of the two
    tie = (low < 7) & (np.take_along_axis(d, np.minimum(low + 1, 7)[:, :, None], 2)[:, :, 0] == best)
    code = np.where(tie & (low % 2 == 1), low + 1, low).astype(np.uint8)
    code = np.where(bad[:, None], 0, code | (np.signbit(x).astype(np.uint8) << 3)).astype(np.uint8)
    return code, np.where(bad, 255, e + 127).astype(np.uint8)


def mxfp4_codes(x):
    """(codes [R, P], scales [R, E]) of rows x [R, K] in value order; P is K rounded up to
    a multiple of 128, E counts blocks up to a multiple of 512; past K both are 0."""
    R, K = x.shape
    own = -(-K // 32) * 32
    P = -(-K // 128) * 128
    full = np.zeros((R, own))
    full[:, :K] = x
    c, e = _block_codes(full.reshape(-1, 32))
    codes, exps = np.zeros((R, P), np.uint8), np.zeros((R, -(-K // 512) * 16), np.uint8)
    codes[:, :own] = c.reshape(R, own)
    exps[:, :own // 32] = e.reshape(R, own // 32)
    return codes, exps


def mxfp4_values(codes, exps, K):
    """What codes [R, P] and scales stand for, the first K of a row, in float64."""
    s = np.where(exps == 255, np.nan, np.ldexp(1.0, exps.astype(np.int64) - 127))
    v = GRID4[codes & 7] * np.where(codes & 8, -1.0, 1.0) * np.repeat(s, 32, axis=1)[:, :codes.shape[1]]
    return v[:, :K]


def mxfp4_rows(codes):
    """The bytes of rows of codes: value 4g + p of a block in nibble g of its word p."""
    R, P = codes.shape
    nib = codes.reshape(R, P // 32, 8, 4).transpose(0, 1, 3, 2).astype(np.uint32)     # [.., p, g]
    words = (nib << (4 * np.arange(8, dtype=np.uint32))).sum(axis=3, dtype=np.uint32)
    return np.ascontiguousarray(words.astype("<u4")).view(np.uint8).reshape(R, P // 2)


def mxfp4_kept_codes(values, cols):
    """(codes [R, cols/2], scales [R, ceil(cols/32)]) of a compressed matrix's values:
    16 kept values have one scale."""
    R, half = values.shape
    own = -(-cols // 32) * 16
    full = np.zeros((R, own))
    full[:, :half] = values
    c, e = _block_codes(full.reshape(-1, 16))
    return c.reshape(R, own)[:, :half], e.reshape(R, own // 16)


def spmm_mxfp4(xv, wv):
    """Y and the sums of magnitudes of the products, in float64."""
    with np.errstate(invalid="ignore"):
        return xv @ wv.T, np.abs(xv) @ np.abs(wv).T
