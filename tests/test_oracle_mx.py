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
