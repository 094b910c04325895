"""Pins of the microscaled formats' oracle: the grids against an independent
implementation of the formats, the rounding's probability, the random words."""
import numpy as np
import pytest
import torch

import oracle
from oracle import mx_ref


def test_grids_are_the_formats():
    codes = torch.arange(128, dtype=torch.uint8)
    e4m3 = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(mx_ref.GRID_M[:127], e4m3[:127]) and np.isnan(e4m3[127])
    # E5M3 without a sign is binary16's upper eight bits below the sign, the top binade taken as numbers
    half = (np.arange(248, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(mx_ref.GRID_V[:248], half) and mx_ref.GRID_V[248] == 65536.0


def test_random_words_start_anywhere_and_differ():
    w = oracle.random_words(1000, 17)
    assert np.array_equal(oracle.random_words(200, 17, first=400), w[400:600])
    assert len(set(w.tolist())) == 1000 and w.max() < 1 << 32
    assert not np.array_equal(oracle.random_words(1000, 18), w)
    assert len({oracle.tensor_seed(5, i) for i in range(1000)}) == 1000
    big = oracle.random_words(1 << 16, oracle.tensor_seed(1, 0)).astype(np.float64) / 2 ** 32
    # 2^16 uniform numbers: mean within five standard deviations, sqrt(1/12) / 2^8
    assert abs(big.mean() - 0.5) < 5 * np.sqrt(1 / 12) / 256
    for bit in range(32):
        ones = ((oracle.random_words(1 << 16, 99) >> np.uint64(bit)) & np.uint64(1)).mean()
        assert abs(ones - 0.5) < 5 * 0.5 / 256, bit


@pytest.mark.parametrize("signed", [True, False])
def test_rounding_keeps_grid_values_and_the_expectation(signed):
    grid, top = (mx_ref.GRID_M, 7) if signed else (mx_ref.GRID_V, 15)
    # values of the grid itself, the block's largest in [2^top, 2^(top+1)): any noise keeps them
    x = np.concatenate([grid[:31], [2.0 ** top]])
    for noise in (0, 2 ** 20 - 1):
        code, exps, value = oracle.moment_codes8(x, np.full(32, noise), grid, top, signed)
        assert np.array_equal(value, x) and exps[0] == 127
    # 3/8 of the way between two codes: five of eight noises round down
    a, b = grid[40], grid[41]
    y = np.full(32, a + 0.375 * (b - a))
    y[0] = 2.0 ** top
    for part in range(8):
        noise = np.full(32, part * 2 ** 17)
        value = oracle.moment_codes8(y, noise, grid, top, signed)[2]
        assert np.all(value[1:] == (b if part >= 5 else a))


def test_blocks_without_values_and_small_ones():
    g, v = mx_ref.GRID_M, mx_ref.GRID_V
    x = np.ones(70)
    x[40] = np.inf
    code, exps, value = oracle.moment_codes8(x, np.zeros(70, int), g, 7, True)
    assert list(exps) == [120, 255, 120] and np.all(code[32:64] == 0) and np.all(np.isnan(value[32:64]))
    assert np.all(value[:32] == 1.0) and np.all(value[64:] == 1.0)
    x = np.full(32, 1e-30)
    x[0] = 1.0                       # far below the block's largest: v keeps a code, m may become zero
    code = oracle.moment_codes8(x, np.zeros(32, int), v, 15, False)[0]
    assert np.all(code[1:] == 1)
    assert np.all(oracle.moment_codes8(x, np.zeros(32, int), g, 7, True)[0][1:] == 0)
    code, exps, value = oracle.moment_codes8(np.zeros(5), np.full(5, 2 ** 20 - 1), g, 7, True)
    assert exps[0] == 0 and not code.any() and not value.any()
    m, vv = oracle.moments8(np.array([0x81, 0x38], np.uint8), np.array([127], np.uint8), np.array([1, 248], np.uint8),
                            np.array([127], np.uint8))
    assert list(m) == [-2.0 ** -9, 1.0] and list(vv) == [2.0 ** -17, 65536.0]


def test_float32_moments_against_exact_fractions():
    from fractions import Fraction
    rng = np.random.default_rng(0)
    g, m = rng.standard_normal(300).astype(np.float32), rng.standard_normal(300).astype(np.float32)
    v = np.abs(rng.standard_normal(300)).astype(np.float32)

    def near(x):                     # float32 nearest to a fraction, ties to even
        f = np.float32(float(x))     # (float(Fraction) rounds once to double; move to the nearest float32 from there)
        c = [np.nextafter(f, np.float32(-np.inf)), f, np.nextafter(f, np.float32(np.inf))]
        d = [abs(Fraction(float(k)) - x) for k in c]
        best = min(d)
        k = [c[i] for i in range(3) if d[i] == best]
        return k[0] if len(k) == 1 else [q for q in k if q.view(np.uint32) % 2 == 0][0]

    b1, o1, b2, o2 = (np.float32(q) for q in (0.9, 1 - 0.9, 0.999, 1 - 0.999))
    F = lambda q: Fraction(float(q))
    mn, vn = oracle.adamw_f32(g, m, v, 0.9, 0.999)
    for i in range(300):
        assert mn[i] == near(F(b1) * F(m[i]) + F(near(F(o1) * F(g[i]))))
        assert vn[i] == near(F(b2) * F(v[i]) + F(near(F(o2) * F(near(F(g[i]) * F(g[i]))))))


def test_4_bit_codes_by_search_and_by_hand():
    # the scale: magnitudes up to 7 units stay, from 7 on the next power of two is taken
    for peak, e in [(6.0, 0), (6.999, 0), (7.0, 1), (8.0, 1), (4.0, 0), (3.5, 0), (3.499, -1), (1.0, -2), (0.0, -127)]:
        x = np.zeros((1, 32))
        x[0, 5] = -peak
        codes, exps = oracle.mxfp4_codes(x)
        assert exps[0, 0] == e + 127 and not exps[0, 1:].any(), peak
        assert codes.shape == (1, 128)
    x = np.zeros((1, 32))
    x[0, :16] = [0, 0.25, 0.2501, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 6.5, -0.25, -0.75, -5.0, 4.0, -0.0]
    want = [0, 0, 0.5, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0, -0.0, -1.0, -4.0, 4.0, -0.0]
    codes, exps = oracle.mxfp4_codes(x)
    got = oracle.mxfp4_values(codes, exps, 16)
    assert exps[0, 0] == 127 and np.array_equal(got[0], want) and np.array_equal(np.signbit(got[0]), np.signbit(want))
    # the nearest value of the format at the block's scale, random blocks
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 96)) * np.exp(rng.standard_normal((50, 96)) * 3)
    codes, exps = oracle.mxfp4_codes(x)
    v = oracle.mxfp4_values(codes, exps, 96)
    s = np.repeat(np.ldexp(1.0, exps.astype(int) - 127), 32, axis=1)[:, :96]
    grid = np.concatenate([mx_ref.GRID4, -mx_ref.GRID4])
    best = np.abs(x[:, :, None] - s[:, :, None] * grid).min(axis=2)
    assert np.array_equal(np.abs(x - v), best)
    assert np.array_equal(mx_ref.GRID4, [0, 0.5, 1, 1.5, 2, 3, 4, 6])
    # blocks without values
    x[3, 40], x[4, 0] = np.nan, np.inf
    codes, exps = oracle.mxfp4_codes(x)
    assert exps[3, 1] == 255 and exps[4, 0] == 255 and not codes[3, 32:64].any()
    v = oracle.mxfp4_values(codes, exps, 96)
    assert np.isnan(v[3, 32:64]).all() and np.isnan(v).sum() == 64


def test_row_bytes_and_kept_codes():
    codes = np.arange(128, dtype=np.uint8).reshape(1, 128) % 16
    rows = oracle.mxfp4_rows(codes)
    words = rows.view("<u4")[0]
    for b in range(4):
        for p in range(4):
            for g in range(8):
                assert (words[4 * b + p] >> (4 * g)) & 15 == codes[0, 32 * b + 4 * g + p]
    # a 2:4 row quantised dense and compressed has the same scales and the same kept codes
    rng = np.random.default_rng(2)
    w = rng.standard_normal((7, 80)).astype(np.float32).view(np.uint32)
    mask, ws = oracle.prune24(w)
    vals, meta, _ = oracle.compress24(w, mask)
    kept, e = oracle.mxfp4_kept_codes(oracle.widen(vals), 80)
    dense, ed = oracle.mxfp4_codes(oracle.widen(ws))
    assert np.array_equal(e, ed[:, :3])
    assert np.array_equal(oracle.decompress24(kept, meta, 80), dense[:, :80] * (mask > 0))


def test_mutations_of_the_4_bit_oracle_would_show():
    """Ties away from zero, a scale by the floor of the exponent, or a saturating 8 change values that the pins hold."""
    x = np.zeros((1, 32))
    x[0, :3] = [7.0, 2.5, 5.0]
    codes, exps = oracle.mxfp4_codes(x)
    assert list(oracle.mxfp4_values(codes, exps, 3)[0]) == [8.0, 2.0, 4.0]
