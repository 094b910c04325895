"""Offsets past 32 bits: rows of activations, codes, outputs and tile chunks that
lie beyond 2^31 elements or bytes, checked where they end."""
import numpy as np
import pytest
import torch

import oracle
import sparse_gemm_02_amd as S

from gpu_util import say

pytestmark = pytest.mark.gpu
LAST = 40


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    S.library()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def f64(t):
    return t.detach().cpu().double().numpy()


def test_norm_codes_and_gradient_past_2_to_31_elements():
    T, K = 300_000, 8192
    say(f"[large norm] {T} x {K}")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    x[-LAST:] = torch.randn((LAST, K), device="cuda", generator=g).bfloat16()
    gamma = (1 + 0.1 * torch.randn(K, device="cuda", generator=g)).bfloat16()
    q, qs = torch.full((T, K), 3, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    S.slope_rmsnorm(x, gamma, 1e-5, Y=y, q=q, q_scale=qs, rstd=rstd)
    torch.cuda.synchronize()
    h = f64(x[-LAST:])
    codes, amax = oracle.row_codes_i8(h * f64(gamma))
    yr, rr = oracle.rmsnorm(h, f64(gamma), 1e-5)
    assert np.array_equal(f64(q[-LAST:]), codes.astype(np.float64)) and not q[:-LAST].any()
    assert np.allclose(f64(qs[-LAST:]), amax / 127 * rr, rtol=2.0 ** -16) and not qs[:-LAST].any()
    assert (np.abs(f64(y[-LAST:]) - yr) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(yr) + 2.0 ** -134).all()
    assert not y[:-LAST].any()
    del q
    dy = torch.zeros_like(x)
    dy[-LAST:] = torch.randn((LAST, K), device="cuda", generator=g).bfloat16()
    dg = torch.empty_like(gamma)
    ws = torch.empty(S.slope_rmsnorm_bwd_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")
    S.slope_rmsnorm_bwd(dy, x, rstd, gamma, y, dg, ws)
    torch.cuda.synchronize()
    d64, r64 = f64(dy[-LAST:]), f64(rstd[-LAST:])
    dxr, dgr = oracle.rmsnorm_bwd(d64, h, r64, f64(gamma))
    a, xh = d64 * f64(gamma), h * r64[:, None]
    terms = r64[:, None] * (np.abs(a) + np.abs(xh) * np.abs(a * xh).mean(axis=1, keepdims=True))
    assert (np.abs(f64(y[-LAST:]) - dxr) <= 2.0 ** -8 * np.abs(dxr) + 2.0 ** -17 * terms + 2.0 ** -134).all()
    assert not y[:-LAST].any()
    # chains of T / groups terms, all but LAST of them zeros
    assert (np.abs(f64(dg) - dgr) <= 2.0 ** -8 * np.abs(dgr) + 2.0 ** -16 * np.abs(d64 * xh).sum(axis=0) + 2.0 ** -134).all()


def _weight(N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.empty((N, K // 2), dtype=torch.bfloat16, device="cuda")
    for a in range(0, N, 50_000):
        v[a:a + 50_000] = 0.02 * torch.randn(v[a:a + 50_000].shape, device="cuda", generator=g)
    meta = torch.full((N, K // 32), 0x44444444, dtype=torch.int32, device="cuda")   # positions 0 and 1 of each four
    packed = torch.empty(S.slope_packed_sparse_i8_bytes(N, K), dtype=torch.uint8, device="cuda")
    ws = torch.empty(N, device="cuda")
    S.slope_pack_sparse_i8(v, meta, N, K, ws, packed)
    return v, meta, packed, ws


@pytest.mark.parametrize("T", [2, 70])
def test_weight_chunks_past_2_to_31_bytes(T):
    N, K = 400_000, 9216
    say(f"[large weight] T={T} N={N} K={K}")
    v, meta, packed, ws = _weight(N, K, 2)
    assert packed.numel() > 1 << 31
    xq = torch.randint(-127, 128, (T, K), dtype=torch.int8, device="cuda")
    xs = torch.rand(T, device="cuda")
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    (S.slope_spmm_i8_decode if T <= 64 else S.slope_spmm_i8_packed)(xq, xs, packed, ws, N, y)
    torch.cuda.synchronize()
    rows = np.r_[0:LAST, N // 2:N // 2 + LAST, N - LAST:N]
    idx = torch.from_numpy(rows).cuda()
    wq = oracle.row_codes_i8(f64(v[idx]))[0]
    ref = oracle.spmm_i8(xq.cpu().numpy(), f64(xs), wq, meta[idx].cpu().numpy().view(np.uint32), K, f64(ws[idx]), "bf16")
    assert np.array_equal(f64(y[:, idx]), ref)


def test_output_past_2_to_31_elements():
    T, K, N = 600_000, 32, 4096
    say(f"[large output] T={T} N={N}")
    v, meta, packed, ws = _weight(N, K, 3)
    xq = torch.randint(-127, 128, (T, K), dtype=torch.int8, device="cuda")
    xs = torch.rand(T, device="cuda")
    y = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    S.slope_spmm_i8_packed(xq, xs, packed, ws, N, y)
    torch.cuda.synchronize()
    wq = oracle.row_codes_i8(f64(v))[0]
    for a in (0, T // 2, T - LAST):
        ref = oracle.spmm_i8(xq[a:a + LAST].cpu().numpy(), f64(xs[a:a + LAST]), wq, meta.cpu().numpy().view(np.uint32), K,
                             f64(ws), "bf16")
        assert np.array_equal(f64(y[a:a + LAST]), ref)
