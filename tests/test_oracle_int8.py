"""Pins of the oracle's RMS norm, its gradient, and the row-scaled int8 codes:
against exact rational arithmetic, central differences and torch's autograd in
float64, and small examples worked by hand."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle


def _code_fraction(u, amax):
    """The integer nearest to 127 u / amax, ties to even, in rational arithmetic."""
    q = 127 * Fraction(float(u)) / Fraction(float(amax))
    k = q.numerator // q.denominator                  # floor
    d = q - k
    return k + (1 if d > Fraction(1, 2) or (d == Fraction(1, 2) and k % 2) else 0)


@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("gfmt", [None, "bf16", "f16", "f32"])
def test_codes_are_the_nearest_integers(fmt, gfmt):
    rng = np.random.default_rng(7)
    u = oracle.round_to(rng.standard_normal((6, 400)), fmt)
    if gfmt:
        u = u * oracle.round_to(1 + 0.1 * rng.standard_normal(400), gfmt)
    q, amax = oracle.row_codes_i8(u)
    for r in range(6):
        assert [_code_fraction(x, amax[r]) for x in u[r]] == q[r].tolist()


def test_codes_at_ties_and_ends():
    # amax 254: the code of x is x / 2, so odd x are ties and go to even codes
    x = np.array([[254.0, 1, 3, 5, -1, -3, 253, -253, -254, 0]])
    q, amax = oracle.row_codes_i8(x)
    assert amax[0] == 254 and q.tolist() == [[127, 0, 2, 2, 0, -2, 126, -126, -127, 0]]
    # amax 127 * 3: ties at 1.5, 4.5, ... of thirds
    q, _ = oracle.row_codes_i8(np.array([[381.0, 1.5, 4.5, -1.5, 1.0, 2.0]]))
    assert q.tolist() == [[127, 0, 2, 0, 0, 1]]


def test_codes_of_empty_and_unbounded_rows():
    q, amax = oracle.row_codes_i8(np.array([[0.0, -0.0], [1.0, np.inf], [np.nan, 1.0], [2.0, 1.0]]))
    assert q.tolist() == [[0, 0], [0, 0], [0, 0], [127, 64]]
    assert amax[0] == 0 and np.isnan(amax[1]) and np.isnan(amax[2]) and amax[3] == 2


def test_rmsnorm_by_hand():
    y, rstd = oracle.rmsnorm(np.array([[3.0, 4.0, 0.0, 0.0]]), np.array([1.0, 2.0, 1.0, 1.0]), 0.0)
    assert rstd[0] == 1 / 2.5 and np.allclose(y, [[1.2, 3.2, 0, 0]], rtol=1e-15)


@pytest.mark.parametrize("with_dh", [False, True])
def test_rmsnorm_bwd_against_autograd_and_differences(with_dh):
    rng = np.random.default_rng(3)
    T, K, eps = 5, 7, 1e-3
    x, g, dy = rng.standard_normal((T, K)), 1 + 0.2 * rng.standard_normal(K), rng.standard_normal((T, K))
    dh = rng.standard_normal((T, K)) if with_dh else None
    _, rstd = oracle.rmsnorm(x, g, eps)
    dx, dg = oracle.rmsnorm_bwd(dy, x, rstd, g, dh)
    tx, tg = torch.tensor(x, requires_grad=True), torch.tensor(g, requires_grad=True)
    y = tx / torch.sqrt((tx * tx).mean(1, keepdim=True) + eps) * tg
    loss = (y * torch.tensor(dy)).sum() + ((tx * torch.tensor(dh)).sum() if with_dh else 0)
    loss.backward()
    assert np.allclose(dx, tx.grad, rtol=1e-12, atol=1e-13) and np.allclose(dg, tg.grad, rtol=1e-12, atol=1e-13)

    def f(x_, g_):
        return (oracle.rmsnorm(x_, g_, eps)[0] * dy).sum() + ((x_ * dh).sum() if with_dh else 0.0)
    # central differences: error h^2 f''' / 6 + 2^-53 |f| / h, below 1e-7 here with h = 1e-5
    for i, j in [(0, 0), (2, 3), (4, 6)]:
        e = np.zeros_like(x)
        e[i, j] = 1e-5
        assert abs((f(x + e, g) - f(x - e, g)) / 2e-5 - dx[i, j]) < 1e-7
    e = np.zeros(K)
    e[2] = 1e-5
    assert abs((f(x, g + e) - f(x, g - e)) / 2e-5 - dg[2]) < 1e-7


def test_spmm_i8_is_the_integer_product():
    rng = np.random.default_rng(5)
    N, K, T = 12, 32, 3
    w = oracle.round_to(rng.standard_normal((N, K)), "f16").astype(np.float16)
    mask, _ = oracle.prune24(w)
    v, meta, _ = oracle.compress24(w, mask)
    q, amax = oracle.row_codes_i8(oracle.widen(v))
    xq = rng.integers(-128, 128, (T, K)).astype(np.int8)
    xs, ws = np.full(T, 0.5), np.full(N, 0.25)
    dense = np.zeros((N, K), np.int64)
    pos = mask.astype(bool)
    dense[pos] = q.reshape(-1)                        # kept values stand in column order within each row
    assert np.array_equal(oracle.spmm_i8(xq, xs, q, meta, K, ws, "f32"), (xq.astype(np.int64) @ dense.T) * 0.125)


def test_residual_sum_rounds_once_to_the_format():
    h = oracle.residual_sum(np.array([[1.0, 1.0, 256.0]]), np.array([[2.0 ** -8, 3 * 2.0 ** -8, 1.0]]), "bf16")
    # 1 + 2^-8 is a tie of bf16 (step 2^-7) and goes to 1; 1 + 3 2^-8 goes to 1 + 2^-6; 257 to 256
    assert h.tolist() == [[1.0, 1 + 2.0 ** -6, 256.0]]
